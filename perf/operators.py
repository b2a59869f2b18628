"""Cases of the operators around the INT8 linear layer: sizes, inputs, calls.

Three operators, each measured as a user's program calls it:

  norm     RMS norm with the residual's addition and INT8 codes with row scales
           as its output (forward), and its backward pass;
  adapter  low-rank adapters of many requests beside one shared INT8 projection:
           the projection with its adapters (forward, down to single tokens), and
           the input and adapter gradients (backward; the projection is frozen);
  adamw    one AdamW step over many tensors, moments held in 32 or in 8 bits.

`own` selects the package's kernels; otherwise `run` computes the same values in
fp32 with elementary torch operations.
"""
import math

import torch

own = False

EPS = 1e-6                      # of the norm
HYPER = dict(lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
SEED = 1234                     # of the stochastic rounding
STEP = 100
BLOCK = 256                     # elements that share one scale of an 8-bit moment
TINY = 2.0 ** -100              # a block whose largest value is below has scale 0

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Three sequences that each decode one token: the norm before a projection.
        dict(name="norm token", op="norm", rows=3, cols=4096, dtype="bf16", had=128, residual=True),
        # A prompt of 2048 tokens at the layer's input width (5376).
        dict(name="norm prompt", op="norm", rows=2048, cols=5376, dtype="bf16", had=128,
             residual=True),
        # A training batch at that width, fp32 residual stream.
        dict(name="norm batch f32", op="norm", rows=12000, cols=5376, dtype="f32", had=128,
             residual=True),
        # The same batch's backward, bf16 stream, fp32 gradient from the dX product.
        dict(name="norm backward", op="norm_bwd", rows=12000, cols=5376, dtype="bf16",
             dn="f32", residual=True),
        # Seven requests with an adapter each decode one token.
        dict(name="adapter token", op="adapter", M=7, K=4096, N=4096, L=12, R=16, w="bf16",
             runs=7),
        # Ragged prompts of nine requests, fp32 adapters of rank 32, the MLP's width.
        dict(name="adapter prompts", op="adapter", M=611, K=4096, N=14336, L=8, R=32, w="f32",
             runs=9),
        # The layer's training batch: 12000 tokens, 5376 -> 7168, three adapters.
        dict(name="adapter batch", op="adapter", M=12000, K=5376, N=7168, L=3, R=16, w="bf16",
             runs=6),
        # Backward of a small ragged batch, fp32 gradient and adapters, rank 64.
        dict(name="adapter backward small", op="adapter_bwd", M=333, K=4096, N=4096, L=5, R=64,
             w="f32", dy="f32", had=64, runs=7),
        # Backward of the training batch.
        dict(name="adapter backward", op="adapter_bwd", M=12000, K=5376, N=7168, L=3, R=16,
             w="bf16", dy="bf16", had=128, runs=6),
        # One block's fp32 adapters and norm weights: 60 ragged tensors.
        dict(name="adamw adapters", op="adamw", tensors=60, elements=2_500_000, p="f32", g="f32",
             bits=32),
        # Dense float parameters of bf16 layers, fp32 moments.
        dict(name="adamw dense", op="adamw", tensors=40, elements=90_000_000, p="bf16", g="bf16",
             bits=32),
        # As many again with their moments in 8 bits.
        dict(name="adamw 8 bit", op="adamw", tensors=70, elements=160_000_000, p="bf16", g="bf16",
             bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, had):
    step = max(16, had)
    return max(1, round(_log(rng, lo, hi) / step)) * step


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "adapter", "adapter_bwd", "adamw"])
    if op == "norm":
        had = rng.choice([0, 16, 64, 128])
        return dict(op=op, rows=_log(rng, 1, 9000), cols=_width(rng, 512, 7168, had),
                    dtype=rng.choice(["f32", "bf16"]), had=had, residual=rng.random() < 0.8)
    if op == "norm_bwd":
        return dict(op=op, rows=_log(rng, 1, 9000), cols=_width(rng, 512, 7168, 0),
                    dtype=rng.choice(["f32", "bf16"]), dn=rng.choice(["f32", "bf16"]),
                    residual=rng.random() < 0.8)
    if op == "adamw":
        bits = rng.choice([8, 32])
        return dict(op=op, tensors=_log(rng, 1, 200), elements=_log(rng, 100_000, 60_000_000),
                    p=rng.choice(["f32", "bf16"]), g=rng.choice(["f32", "bf16"]), bits=bits)
    case = dict(op=op, M=_log(rng, 1, 4000), K=_width(rng, 1024, 5376, 128),
                N=_width(rng, 1024, 7168, 0), L=rng.randint(1, 16),
                R=8 * rng.randint(1, 8), w=rng.choice(["f32", "bf16"]))
    case["runs"] = min(case["M"], rng.randint(1, 20))
    if op == "adapter_bwd":
        case["dy"] = rng.choice(["f32", "bf16"])
        case["had"] = rng.choice([0, 16, 64, 128])
    return case


def work(c):
    op = c["op"]
    if op == "norm":
        n, e = c["rows"] * c["cols"], BYTES[c["dtype"]]
        return {"bytes": n * (e + (2 * e if c["residual"] else 0) + 1 + 2) + 4 * c["cols"]
                + 8 * c["rows"], "flops": 0}
    if op == "norm_bwd":
        n, e = c["rows"] * c["cols"], BYTES[c["dtype"]]
        return {"bytes": n * (BYTES[c["dn"]] + (3 if c["residual"] else 2) * e) + 8 * c["cols"]
                + 4 * c["rows"], "flops": 0}
    if op == "adamw":
        state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": c["elements"] * (2 * BYTES[c["p"]] + BYTES[c["g"]] + state), "flops": 0}
    M, K, N, L, R = (c[k] for k in "MKNLR")
    used = min(L, c["runs"])
    lowrank = used * R * (K + N)
    if op == "adapter":
        return {"bytes": M * K + N * K + 4 * M * N + lowrank * BYTES[c["w"]] + 4 * M * R + 8 * M
                + 8 * N, "flops": 2 * M * N * K + 2 * M * R * (K + N)}
    return {"bytes": M * N * (BYTES[c["dy"]] + 1) + M * K * 5 + N * K + 4 * M * R
            + lowrank * BYTES[c["w"]] + 4 * L * R * (K + N) + 12 * M,
            "flops": 2 * M * N * K + 4 * M * R * (K + N)}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _activations(rows, cols, g, std, dtype):
    """Normal values, one channel in a hundred eight times larger, and the last
    rows of a larger batch empty, as padding leaves them."""
    x = _randn((rows, cols), g, std)
    x[:, torch.randperm(cols, generator=g, device="cuda")[:cols // 100]] *= 8.0
    if rows >= 64:
        x[rows - rows // 64:] = 0.0
    return x.to(dtype)


def _codes(rows, cols, g):
    """INT8 codes with row scales, as the quantizers give them for normal rows."""
    q = (torch.randn((rows, cols), generator=g, device="cuda") * 32).round_().clamp_(-127, 127)
    return q.to(torch.int8), (torch.rand(rows, generator=g, device="cuda") + 0.5) * 0.03


def _quantize(g):
    a = g.abs().amax(1, keepdim=True)
    s = a / 127.0
    return torch.where(a > 0, g / s, 0.0).round().to(torch.int8), s.squeeze(1)


def _request_ids(M, L, runs, seed):
    """Adapter of each token: `runs` requests of ragged lengths one after another,
    each with one of L adapters, now and then with none (-1)."""
    import random
    r = random.Random(seed)
    cuts = sorted(r.sample(range(1, M), min(runs, M) - 1)) if M > 1 else []
    ids, pick = [], list(range(L))
    r.shuffle(pick)
    for k, (a, b) in enumerate(zip([0] + cuts, cuts + [M])):
        ids += [-1 if k % 6 == 5 else pick[k % L]] * (b - a)
    return torch.tensor(ids, dtype=torch.int32, device="cuda")


def _sizes(tensors, elements):
    """Ragged tensor sizes with the given sum, the same for every seed: most of them
    small, a few large."""
    import random
    r = random.Random(tensors)
    share = [math.exp(r.uniform(0, 5)) for _ in range(tensors)]
    sizes = [max(1, int(elements * s / sum(share))) for s in share]
    sizes[0] += elements - sum(sizes)
    return sizes


def prepare(case, seed):
    c, g = case, _gen(seed)
    dev = "cuda"
    s = dict(case)
    if c["op"] in ("norm", "norm_bwd"):
        rows, cols, dt = c["rows"], c["cols"], DTYPES[c["dtype"]]
        s["gamma"] = 1.0 + _randn((cols,), g, 0.1)
        s["out_h"] = torch.empty((rows, cols), dtype=dt, device=dev)
        if c["op"] == "norm":
            s["x"] = _activations(rows, cols, g, 1.0, dt)
            s["res"] = _activations(rows, cols, g, 2.0, dt) if c["residual"] else None
            s["out_q"] = torch.empty((rows, cols), dtype=torch.int8, device=dev)
            s["out_y"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
            s["out_s"] = torch.empty((rows,), device=dev)
            s["out_rstd"] = torch.empty((rows,), device=dev)
            return s
        s["h"] = _activations(rows, cols, g, 2.0, dt)
        s["out_dgamma"] = torch.empty((cols,), device=dev)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dn"] = _randn((rows, cols), g, 0.01, DTYPES[c["dn"]])
        s["dres"] = _randn((rows, cols), g, 0.01, dt) if c["residual"] else None
        if own:     # the scratch memory that a training program keeps
            import w8a8_integer_linear_amd as qlin
            s["ws"] = torch.empty(qlin.qlin_rmsnorm_bwd_ws_bytes(rows, cols), dtype=torch.uint8,
                                  device=dev)
        return s
    if c["op"] in ("adapter", "adapter_bwd"):
        M, K, N, L, R = (c[k] for k in "MKNLR")
        s["qx"], s["sx"] = _codes(M, K, g)
        s["qw"], s["sw"] = _codes(N, K, g)
        s["sw"] *= 0.02
        s["a"] = _randn((L, R, K), g, 1.0 / math.sqrt(K), DTYPES[c["w"]])
        s["b"] = _randn((L, N, R), g, 0.05, DTYPES[c["w"]])
        s["scale"] = torch.rand(L, generator=g, device=dev) + 0.5
        s["ids"] = _request_ids(M, L, c["runs"], seed)
        if c["op"] == "adapter":
            s["bias"] = _randn((N,), g, 0.01)
            s["out_y"] = torch.empty((M, N), device=dev)
            s["out_u"] = torch.empty((M, R), device=dev)
        else:
            s["dy"] = _randn((M, N), g, 0.01, DTYPES[c["dy"]])
            s["qg"], s["sg"] = _quantize(s["dy"].float() * s["sw"])
            s["u"] = _adapter_u(s)
            s["out_dx"] = torch.empty((M, K), device=dev)
            s["out_da"] = torch.empty((L, R, K), device=dev)
            s["out_db"] = torch.empty((L, N, R), device=dev)
            s["out_order"] = torch.empty((M,), dtype=torch.int32, device=dev)
            s["out_start"] = torch.empty((L + 1,), dtype=torch.int32, device=dev)
        if own:     # the workspace that a program keeps between calls
            import w8a8_integer_linear_amd as qlin
            size = (qlin.qlin_adapter_fwd_ws_bytes if c["op"] == "adapter"
                    else qlin.qlin_adapter_bwd_ws_bytes)(M, N, K, L, R)
            s["ws"] = torch.zeros(size, dtype=torch.uint8, device=dev)
        return s
    # adamw: the tensors lie in flat buffers, each at a multiple of BLOCK elements.
    sizes = _sizes(c["tensors"], c["elements"])
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    live = torch.zeros(at, dtype=torch.bool, device=dev)
    decay = torch.zeros(at // BLOCK, device=dev)
    decays = [HYPER["weight_decay"] if k % 3 else 0.0 for k in range(len(sizes))]
    for n, a, wd in zip(sizes, starts, decays):
        live[a:a + n] = True
        decay[a // BLOCK:-(-(a + n) // BLOCK)] = wd
    s["decay"] = decay
    s["p"] = (_randn((at,), g, 0.02) * live).to(DTYPES[c["p"]])
    s["grad"] = (_randn((at,), g, 1e-3) * live).to(DTYPES[c["g"]])
    m = _randn((at,), g, 5e-4) * live
    r = (_randn((at,), g, 5e-4).abs_() + 5e-4) * live
    if c["bits"] == 32:
        s["m"], s["v"] = m, r.square_()
        s["ms"] = s["vs"] = None
    else:
        s["m"], s["ms"] = _eight(m)
        s["v"], s["vs"] = _eight(r)
    if own:         # the plan: where the tensors are, built once by a program
        import w8a8_integer_linear_amd as qlin
        part = lambda t, a, n: None if t is None else t[a:a + n]                    # noqa: E731
        scales = lambda t, a, n: None if t is None else t[a // BLOCK:-(-(a + n) // BLOCK)]  # noqa: E731
        s["plan"] = qlin.qlin_adamw_tensors_plan([
            dict(p=part(s["p"], a, n), g=part(s["grad"], a, n), m=part(s["m"], a, n),
                 v=part(s["v"], a, n), m_scale=scales(s["ms"], a, n),
                 v_scale=scales(s["vs"], a, n), weight_decay=wd, index0=a)
            for n, a, wd in zip(sizes, starts, decays)])
    return s


def _eight(t):
    """e4m3 codes of blocks of BLOCK values, with a scale each."""
    t = t.view(-1, BLOCK)
    a = t.abs().amax(1, keepdim=True)
    inv = torch.where(a >= TINY, 448.0 / a, 0.0)
    code = (t * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return code.view(-1), torch.where(a >= TINY, a / 448.0, 0.0).view(-1)


# ----------------------------------------------------------- plain forms

def _hadamard(n, dtype=torch.float32):
    h = torch.ones((1, 1), dtype=dtype, device="cuda")
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(n)


def _rotate(t, had):
    if not had:
        return t
    return (t.reshape(-1, had) @ _hadamard(had, t.dtype)).reshape(t.shape)


def _norm(s):
    h = s["x"]
    if s["res"] is not None:
        h = (s["x"].float() + s["res"].float()).to(h.dtype)
    f = h.float()
    rstd = 1.0 / torch.sqrt(f.square().mean(1) + EPS)
    n = _rotate(f * rstd[:, None] * s["gamma"], s["had"])
    q, sc = _quantize(n)
    return [h, rstd, sc, (q.float() * sc[:, None]).to(torch.bfloat16)]


def _norm_bwd(s):
    xh = s["h"].float() * s["rstd"][:, None]
    dn = s["dn"].float()
    g = dn * s["gamma"]
    dh = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return [dh.to(s["h"].dtype), (dn * xh).sum(0)]


def _of_own_adapter(t, ids):
    """[M, L, R] with every adapter's values but the token's own replaced by zeros."""
    mine = ids[:, None] == torch.arange(t.shape[1], device=t.device)
    return torch.where(mine[:, :, None], t, 0.0)


def _adapter_u(s):
    """[M, R]: scale (x^ A^T) of each token's own adapter."""
    L, R, K = s["a"].shape
    x = s["qx"].float() * s["sx"][:, None]
    every = (x @ s["a"].float().reshape(L * R, K).T).view(-1, L, R) * s["scale"][:, None]
    return _of_own_adapter(every, s["ids"]).sum(1)


def _adapter(s):
    L, R, K = s["a"].shape
    M = s["qx"].shape[0]
    u = _adapter_u(s)
    y = (s["qx"].float() @ s["qw"].float().T) * s["sx"][:, None] * s["sw"] + s["bias"]
    spread = _of_own_adapter(u[:, None, :].expand(M, L, R), s["ids"]).reshape(M, L * R)
    y += spread @ s["b"].float().transpose(1, 2).reshape(L * R, -1)
    return [y, u]


def _adapter_bwd(s):
    L, R, K = s["a"].shape
    M, N = s["dy"].shape
    dy = s["dy"].float()
    bt = s["b"].float().transpose(1, 2).reshape(L * R, N)
    v = _of_own_adapter((dy @ bt.T).view(M, L, R) * s["scale"][:, None], s["ids"])
    v = v.reshape(M, L * R)
    dx = (s["qg"].float() @ s["qw"].float()) * s["sg"][:, None]
    dx = _rotate(dx + v @ s["a"].float().reshape(L * R, K), s["had"])
    u = _of_own_adapter(s["u"][:, None, :].expand(M, L, R), s["ids"]).reshape(M, L * R)
    x = s["qx"].float() * s["sx"][:, None]
    da = (v.T @ x).view(L, R, K)
    db = (u.T @ dy).view(L, R, N).transpose(1, 2).contiguous()
    return [dx, da, db]


def _philox16(count, seed, step, stream):
    """The 16-bit uniforms of elements 0 .. count - 1 (Philox4x32-10, Salmon et al.
    2011): half (i & 1) of word (i & 7) >> 1 at counter (i >> 3, step), key seed;
    `stream` is added to the counter's highest word."""
    m32 = 0xFFFFFFFF
    i = torch.arange(count // 8, device="cuda")
    c = [i & m32, i >> 32, torch.full_like(i, step & m32), torch.full_like(i, (step >> 32) + stream)]
    k0, k1 = seed & m32, seed >> 32

    def product(x, m):      # high and low words of a 32 x 32 bit product
        lo, hi = x * (m & 0xFFFF), x * (m >> 16)
        mid = (lo >> 16) + (hi & 0xFFFF)
        return (hi >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)

    for _ in range(10):
        h0, l0 = product(c[0], 0xD2511F53)
        h1, l1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    words = torch.stack(c, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(-1).to(torch.int32)


def _adam_consts():
    h, t = HYPER, STEP
    return (1 - h["beta1"], 1 - h["beta2"], h["lr"] / (1 - h["beta1"] ** t),
            1 / math.sqrt(1 - h["beta2"] ** t))


def _adamw(s):
    b1, b2, eps = HYPER["beta1"], HYPER["beta2"], HYPER["eps"]
    a1, a2, c1, c2 = _adam_consts()
    eight = s["bits"] == 8
    p, g = s["p"].float().view(-1, BLOCK), s["grad"].float().view(-1, BLOCK)
    m, v = s["m"].float().view(-1, BLOCK), s["v"].float().view(-1, BLOCK)
    if eight:
        m, v = m * s["ms"][:, None], (v * s["vs"][:, None]).square()
    m = b1 * m + a1 * g
    v = b2 * v + (a2 * g) * g
    r = torch.sqrt(v)
    p = p * (1.0 - HYPER["lr"] * s["decay"])[:, None] - c1 * (m / (r * c2 + eps))
    if s["p"].dtype == torch.float32:
        s["p"].copy_(p.view(-1))
    else:           # bf16 parameters are rounded stochastically
        bits = p.view(torch.int32) + _philox16(p.numel(), SEED, STEP, 1 << 31).view(p.shape)
        s["p"].copy_((bits & ~0xFFFF).view(torch.float32).view(-1))
    if not eight:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
        return [s["p"], s["m"], s["v"]]
    code, ms = _eight(m.view(-1))
    s["m"].copy_(code)
    s["ms"].copy_(ms)
    # The root of the second moment, rounded stochastically to e4m3; a value above
    # zero never becomes zero.
    a = r.amax(1, keepdim=True)
    t = (r * torch.where(a >= TINY, 448.0 / a, 0.0)).clamp(max=448.0)
    low = torch.where(t < 2.0 ** -6, 2.0 ** -6, 0.0)
    bits = (t + low).view(torch.int32) + (_philox16(t.numel(), SEED, STEP, 0) << 4).view(t.shape)
    near = (bits & ~0xFFFFF).view(torch.float32) - low
    near = torch.where(t > 0, near.clamp(min=2.0 ** -9), near)
    s["v"].copy_(near.view(-1).to(torch.float8_e4m3fn))
    s["vs"].copy_(torch.where(a >= TINY, a / 448.0, 0.0).view(-1))
    return [s["p"], s["m"], s["v"], s["ms"], s["vs"]]


PLAIN = {"norm": _norm, "norm_bwd": _norm_bwd, "adapter": _adapter, "adapter_bwd": _adapter_bwd,
         "adamw": _adamw}


# -------------------------------------------------------------------- run

def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    import w8a8_integer_linear_amd as qlin
    if s["op"] == "norm":
        _, sc, h, rstd, y = qlin.qlin_rmsnorm_quant(
            s["x"], s["gamma"], EPS, residual=s["res"], had_block=s["had"], h=s["out_h"],
            q=s["out_q"], s=s["out_s"], rstd=s["out_rstd"], y=s["out_y"])
        return [h, rstd, sc, y]
    if s["op"] == "norm_bwd":
        dh, dgamma = qlin.qlin_rmsnorm_bwd(s["dn"], s["h"], s["rstd"], s["gamma"], dres=s["dres"],
                                           dh=s["out_h"], dgamma=s["out_dgamma"],
                                           workspace=s["ws"])
        return [dh, dgamma]
    if s["op"] == "adapter":
        y, u = qlin.qlin_adapter_fwd(s["qx"], s["sx"], s["qw"], s["sw"], s["a"], s["b"],
                                     s["scale"], s["ids"], bias=s["bias"], y=s["out_y"],
                                     u=s["out_u"], workspace=s["ws"])
        return [y, u]
    if s["op"] == "adapter_bwd":
        order, start = qlin.qlin_adapter_group(s["ids"], s["a"].shape[0], order=s["out_order"],
                                               start=s["out_start"])
        dx, da, db = qlin.qlin_adapter_bwd(
            s["dy"], s["qg"], s["sg"], s["qw"], s["qx"], s["sx"], s["u"], s["a"], s["b"],
            s["scale"], s["ids"], order, start, had_block=s["had"], dx=s["out_dx"],
            da=s["out_da"], db=s["out_db"], workspace=s["ws"])
        return [dx, da, db]
    qlin.qlin_adamw_tensors(s["plan"], HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"],
                            SEED, STEP)
    out = [s["p"], s["m"], s["v"]]
    return out if s["bits"] == 32 else out + [s["ms"], s["vs"]]


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The operator's definition in 64 bits (codes and stochastically rounded
    values as the numbers that are rounded)."""
    s = prepare(case, seed)
    d = torch.float64
    op = case["op"]
    if op == "norm":
        h = s["x"].to(d)
        if s["res"] is not None:
            h = (h + s["res"].to(d)).to(s["x"].dtype).to(d)     # the stream's own type
        rstd = (h.pow(2).sum(1) / h.shape[1] + EPS).pow(-0.5)
        n = h * rstd.unsqueeze(1) * s["gamma"].to(d)
        if case["had"]:
            k = case["had"]
            n = torch.matmul(n.view(-1, k), _hadamard(k, d)).view(n.shape)
        sc = n.abs().max(1).values / 127
        q = torch.round(n / torch.where(sc > 0, sc, 1).unsqueeze(1))
        return [h, rstd, sc, q * sc.unsqueeze(1)]
    if op == "norm_bwd":
        h, dn = s["h"].to(d), s["dn"].to(d)
        r, w = s["rstd"].to(d).unsqueeze(1), s["gamma"].to(d)
        # d/dh of sum(dn * h * r(h) * w), r's own derivative being -r^3 h / cols
        dh = dn * w * r - h * r.pow(3) * ((dn * w * h).sum(1, keepdim=True) / h.shape[1])
        if s["dres"] is not None:
            dh = dh + s["dres"].to(d)
        return [dh, (dn * h * r).sum(0)]
    if op in ("adapter", "adapter_bwd"):
        x = s["qx"].to(d) * s["sx"].to(d).unsqueeze(1)
        a, b, sc = s["a"].to(d), s["b"].to(d), s["scale"].to(d)
        M, R = x.shape[0], a.shape[1]
        rows = [torch.nonzero(s["ids"] == k).squeeze(1) for k in range(a.shape[0])]
        if op == "adapter":
            y = torch.matmul(x, (s["qw"].to(d) * s["sw"].to(d).unsqueeze(1)).t()) + s["bias"].to(d)
            u = torch.zeros(M, R, dtype=d, device="cuda")
            for k, at in enumerate(rows):
                u[at] = sc[k] * torch.matmul(x[at], a[k].t())
                y[at] += torch.matmul(u[at], b[k].t())
            return [y, u]
        dy, u = s["dy"].to(d), s["u"].to(d)
        dx = torch.matmul(s["qg"].to(d) * s["sg"].to(d).unsqueeze(1), s["qw"].to(d))
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for k, at in enumerate(rows):
            v = sc[k] * torch.matmul(dy[at], b[k])
            dx[at] += torch.matmul(v, a[k])
            da[k] = torch.matmul(v.t(), x[at])
            db[k] = torch.matmul(dy[at].t(), u[at])
        if case["had"]:
            k = case["had"]
            dx = torch.matmul(dx.view(-1, k), _hadamard(k, d)).view(dx.shape)
        return [dx, da, db]
    lr, b1, b2 = HYPER["lr"], HYPER["beta1"], HYPER["beta2"]
    m, v, g = s["m"].to(d), s["v"].to(d), s["grad"].to(d)
    if case["bits"] == 8:
        m = (m.view(-1, BLOCK) * s["ms"].to(d).unsqueeze(1)).view(-1)
        v = (v.view(-1, BLOCK) * s["vs"].to(d).unsqueeze(1)).view(-1) ** 2
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    wd = s["decay"].to(d).repeat_interleave(BLOCK)
    p = s["p"].to(d)
    p = p - lr * wd * p - lr * (m / (1 - b1 ** STEP)) / (torch.sqrt(v / (1 - b2 ** STEP))
                                                        + HYPER["eps"])
    if case["bits"] == 32:
        return [p, m, v]
    out = []
    for t in (m, torch.sqrt(v)):
        top = t.view(-1, BLOCK).abs().max(1).values
        t = t.view(-1, BLOCK) * (448 / torch.where(top > 0, top, 1)).unsqueeze(1)
        out.append((t.view(-1), top / 448))
    return [p, out[0][0], out[1][0], out[0][1], out[1][1]]
