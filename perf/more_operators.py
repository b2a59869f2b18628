"""Cases of the operators inside a feed-forward block: sizes, inputs, calls.

Between the block's two projections stand an activation, mostly a gate, and in
training what the backward pass needs of them.  Three operators:

  act        an INT8 product with bias, activation and residual in its epilogue;
  gated      both projections of a gated block in one product, with the activation
             of the one and the product with the other in its epilogue;
  act_bwd    the backward of either from a checkpoint of z (the products before the
             activation) in 8 bits: dz, its sums over the tokens (the bias's gradient)
             and the scales of its two quantizations.

`train` runs act or gated with the checkpoint kept, and act_bwd on it.  The checkpoint
holds INT8 codes of z with a scale for each 32 outputs of a row.

`own` selects the package's kernels; otherwise `run` computes the same values with
elementary torch operations.
"""
import math

import torch

own = False

BLOCK = 32                      # outputs of a row that share a scale of the checkpoint
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
ROOT = math.sqrt(2 / math.pi)   # of the tanh form of GELU
CUBE = 0.044715


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Three requests that each decode one token through a gated block's first half.
        dict(name="gated token", op="gated", M=3, K=4096, F=14336, act="silu", y="bf16",
             bias=False),
        # Ragged prompts of together 611 tokens.
        dict(name="gated prompt", op="gated", M=611, K=4096, F=14336, act="silu", y="bf16",
             bias=False),
        # The MLP's training batch, evaluated: 8192 tokens, nothing kept.
        dict(name="gated batch", op="gated", M=8192, K=4096, F=14336, act="gelu_tanh", y="bf16",
             bias=True),
        # A training step's way through the gate and back, 2048 tokens of the layer's width.
        dict(name="gated train", op="train", gated=True, M=2048, K=5376, F=7168, act="silu",
             y="bf16", dy="f32", dz="bf16", bias=False),
        # Backward of a small ragged batch in fp32 throughout, an odd width.
        dict(name="gated backward small", op="act_bwd", gated=True, M=333, F=1808,
             act="gelu_tanh", dy="f32", dz="f32"),
        # Backward of the MLP's training batch; dy comes from the second projection's dX.
        dict(name="gated backward", op="act_bwd", gated=True, M=8192, F=14336, act="silu",
             dy="f32", dz="bf16"),
        # The block's second half for five tokens: back to the width, onto the residual stream.
        dict(name="act token", op="act", M=5, K=14336, F=4096, act="none", y="bf16",
             residual="bf16", bias=True),
        # The first half of a block without a gate, ragged prompts, fp32.
        dict(name="act prompt", op="act", M=777, K=4096, F=14336, act="gelu", y="f32",
             residual=None, bias=True),
        # The layer's training batch onto a residual stream in fp32.
        dict(name="act batch", op="act", M=12000, K=5376, F=7168, act="none", y="f32",
             residual="f32", bias=True),
        # The MLP with GELU, half a batch, forward with its checkpoint and back.
        dict(name="act train", op="train", gated=False, M=4000, K=4096, F=14336, act="gelu",
             y="bf16", dy="f32", dz="bf16", bias=True),
        # Backward of a short batch, fp32.
        dict(name="act backward small", op="act_bwd", gated=False, M=100, F=4096, act="relu",
             dy="f32", dz="f32"),
        # Backward of the layer's training batch, a bf16 stream.
        dict(name="act backward", op="act_bwd", gated=False, M=12000, F=7168, act="gelu",
             dy="bf16", dz="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(1, round(_log(rng, lo, hi) / 16)) * 16


def draw(rng):
    op = rng.choice(["act", "gated", "act_bwd", "train"])
    case = dict(op=op, M=_log(rng, 1, 9000 if op == "act_bwd" else 4000), F=_width(rng, 512, 7168),
                act=rng.choice(["relu", "silu", "gelu", "gelu_tanh"]))
    if op in ("act_bwd", "train"):
        case["gated"] = rng.random() < 0.5
        case["dy"] = rng.choice(["f32", "bf16"])
        case["dz"] = rng.choice(["f32", "bf16"])
    if op != "act_bwd":
        case["K"] = _width(rng, 1024, 5376)
        case["y"] = rng.choice(["f32", "bf16"])
        case["bias"] = rng.random() < 0.5
    if op == "act":
        case["act"] = rng.choice(["none", case["act"]])
        case["residual"] = rng.choice([None, "f32", "bf16"])
    return case


def _outputs(c):
    """Rows of the weight: gate and up, or the projection's own."""
    return 2 * c["F"] if c["op"] == "gated" or c.get("gated") else c["F"]


def _blocks(c):
    return _outputs(c) // c["F"] * -(-c["F"] // BLOCK)


def work(c):
    M, F, N = c["M"], c["F"], _outputs(c)
    held = M * N + 4 * M * _blocks(c)
    back = M * F * BYTES[c.get("dy", "f32")] + M * N * BYTES[c.get("dz", "f32")] + 8 * M + 12 * N
    if c["op"] == "act_bwd":
        return {"bytes": held + back, "flops": 0}
    K = c["K"]
    n = M * K + N * K + 4 * M + 4 * N + M * F * BYTES[c["y"]] + (4 * N if c["bias"] else 0)
    if c.get("residual"):
        n += M * F * BYTES[c["residual"]]
    if c["op"] == "train":
        # (The checkpoint is written and read: it outlives the forward pass.)
        n += 2 * held + back
    return {"bytes": n, "flops": 2 * M * N * K}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _codes(rows, cols, g):
    """INT8 codes with row scales, as the quantizers give them for normal rows."""
    q = (torch.randn((rows, cols), generator=g, device="cuda") * 32).round_().clamp_(-127, 127)
    return q.to(torch.int8), torch.rand(rows, generator=g, device="cuda") + 0.5


def prepare(case, seed):
    c, g, dev = case, _gen(seed), "cuda"
    s = dict(case)
    M, F, N = c["M"], c["F"], _outputs(c)
    gated = N != F
    pad = M // 64           # the last rows of a larger batch are empty, as padding leaves them
    s["sx"] = (torch.rand(M, generator=g, device=dev) + 0.5) * 0.03
    if c["op"] != "act_bwd":
        K = c["K"]
        s["qx"], _ = _codes(M, K, g)
        s["qw"], s["sw"] = _codes(N, K, g)
        s["sw"] *= 1.5 / (math.sqrt(K) * 32 * 32 * 0.03)       # z is of the order of one
        s["qx"][M - pad:] = 0
        s["bias"] = _randn((N,), g, 0.1) if c["bias"] else None
        r = c.get("residual")
        s["res"] = _randn((M, F), g, 2.0, DTYPES[r]) if r else None
        s["out_y"] = torch.empty((M, F), dtype=DTYPES[c["y"]], device=dev)
    else:
        s["sw"] = (torch.rand(N, generator=g, device=dev) + 0.5) * 1e-3
        z = _randn((M, N), g, 1.5)
        z[:, torch.randperm(N, generator=g, device=dev)[:N // 100]] *= 4.0
        s["ck"], s["ck_s"] = _checkpoint(z, F)
    s["sx"][M - pad:] = 0
    if c["op"] in ("act_bwd", "train"):
        s["dy"] = _randn((M, F), g, 0.01)
        s["dy"][M - pad:] = 0
        s["dy"] = s["dy"].to(DTYPES[c["dy"]])
        s["out_dz"] = torch.empty((M, N), dtype=DTYPES[c["dz"]], device=dev)
        s["out_s1"] = torch.empty((M,), device=dev)
        s["out_s2"] = torch.empty((N,), device=dev)
        s["out_db"] = torch.empty((N,), device=dev)
    if c["op"] == "train":
        s["out_ck"] = torch.empty((M, N), dtype=torch.int8, device=dev)
        s["out_ck_s"] = torch.empty((M, _blocks(c)), device=dev)
    if own:     # the scratch memory that a program keeps between calls
        import w8a8_integer_linear_amd as qlin
        if c["op"] != "act_bwd":
            size = (qlin.qlin_fwd_gated_ws_bytes if gated else qlin.qlin_fwd_act_ws_bytes)(M, F, K)
            s["ws"] = torch.zeros(size, dtype=torch.uint8, device=dev)
        if c["op"] != "act" and c["op"] != "gated":
            s["bwd_ws"] = torch.empty(qlin.qlin_act_bwd_ws_bytes(M, F, gated), dtype=torch.uint8,
                                      device=dev)
    return s


# ----------------------------------------------------------- plain forms

def _in_blocks(z, F):
    """[M, halves, blocks, BLOCK], each half filled up to whole blocks with zeros."""
    z = z.view(z.shape[0], -1, F)
    z = torch.nn.functional.pad(z, (0, -F % BLOCK))
    return z.view(z.shape[0], z.shape[1], -1, BLOCK)


def _checkpoint(z, F):
    """INT8 codes of z [M, N], N = F or 2 F, and a scale per block."""
    b = _in_blocks(z, F)
    # (By a tensor: torch multiplies by the rounded reciprocal of a number.)
    s = b.abs().amax(3) / torch.full((), 127.0, dtype=z.dtype, device=z.device)
    q = torch.where(s[..., None] > 0, b / s[..., None], 0.0).round().to(torch.int8)
    return q.view(*q.shape[:2], -1)[:, :, :F].reshape(z.shape), s.view(z.shape[0], -1)


def _restored(q, s, F):
    each = s.view(s.shape[0], q.shape[1] // F, -1).repeat_interleave(BLOCK, 2)[:, :, :F]
    return q.float() * each.reshape(q.shape)


def _z(s, whole):
    """Products with their scales and bias.  whole: the integer sums to their last
    digit, which decides on the codes of values next to a border; their size passes
    the 24 bits of a 32-bit float."""
    d = torch.float64 if whole else torch.float32
    acc = (s["qx"].to(d) @ s["qw"].to(d).T).float()
    z = acc * s["sx"][:, None] * s["sw"]
    return z if s["bias"] is None else z + s["bias"]


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(ROOT * (z + CUBE * z * z * z)))


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        density = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * density
    t = torch.tanh(ROOT * (z + CUBE * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * ROOT * (1.0 + 3 * CUBE * z * z)


def _forward(s, z):
    F = s["F"]
    y = _act(z[:, :F], s["act"])
    if z.shape[1] != F:
        y = y * z[:, F:]
    if s.get("res") is not None:
        y = y + s["res"].float()
    return y.to(DTYPES[s["y"]])


def _backward(s, ck, ck_s):
    F = s["F"]
    z, dy = _restored(ck, ck_s, F), s["dy"].float()
    dz = dy * _slope(z[:, :F], s["act"])
    if z.shape[1] != F:
        dz = torch.cat([dz * z[:, F:], dy * _act(z[:, :F], s["act"])], 1)
    s1 = (dz * s["sw"]).abs().amax(1) / 127.0
    s2 = (dz * s["sx"][:, None]).abs().amax(0) / 127.0
    return [dz.to(DTYPES[s["dz"]]), s1, s2, dz.sum(0)]


# -------------------------------------------------------------------- run

def run(s):
    op = s["op"]
    if not own:
        if op == "act_bwd":
            return _backward(s, s["ck"], s["ck_s"])
        z = _z(s, whole=op == "train")
        y = [_forward(s, z)]
        return y if op != "train" else y + _backward(s, *_checkpoint(z, s["F"]))
    import w8a8_integer_linear_amd as qlin
    gated = op == "gated" or s.get("gated", False)
    out, ck, ck_s = [], s.get("ck"), s.get("ck_s")
    if op != "act_bwd":
        given = dict(bias=s["bias"], act=s["act"], y=s["out_y"], ck=s.get("out_ck"),
                     ck_s=s.get("out_ck_s"), workspace=s["ws"])
        if gated:
            y, ck, ck_s = qlin.qlin_fwd_gated(s["qx"], s["sx"], s["qw"], s["sw"], **given)
        else:
            y, ck, ck_s = qlin.qlin_fwd_act(s["qx"], s["sx"], s["qw"], s["sw"], residual=s["res"],
                                            **given)
        out = [y]
    if op in ("act_bwd", "train"):
        # (The prepared codes are a view where an ungated width ends inside a block.)
        out += qlin.qlin_act_bwd(s["dy"], ck.contiguous(), ck_s, s["act"], gated=gated, sw=s["sw"],
                                 sx=s["sx"], dz=s["out_dz"], s1=s["out_s1"], s2=s["out_s2"],
                                 db=s["out_db"], workspace=s["bwd_ws"])
    return out


# ------------------------------------------------------------------ exact

def _value_and_slope(z, act):
    """act(z) and its derivative in 64 bits, through the logistic function and the
    normal distribution's."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
    inner, rate = z, 1.0
    if act == "gelu_tanh":      # (1 + tanh t) / 2 is the logistic function of 2 t
        inner, rate = 2 * ROOT * (z + CUBE * z.pow(3)), 2 * ROOT * (1 + 3 * CUBE * z.square())
    p = torch.sigmoid(inner)
    return z * p, p + z * p * torch.sigmoid(-inner) * rate


def exact(case, seed):
    """The operator's definition in 64 bits."""
    s = prepare(case, seed)
    d, F, N, op = torch.float64, case["F"], _outputs(case), case["op"]
    out = []
    if op == "act_bwd":
        q, sc = s["ck"].to(d), s["ck_s"].to(d)
        b = _in_blocks(q, F)
        z = (b * sc.view(*b.shape[:3], 1)).reshape(b.shape[0], b.shape[1], -1)[:, :, :F].reshape(q.shape)
    else:
        z = torch.matmul(s["qx"].to(d) * s["sx"].to(d).unsqueeze(1),
                         (s["qw"].to(d) * s["sw"].to(d).unsqueeze(1)).t())
        if s["bias"] is not None:
            z += s["bias"].to(d)
        y = _value_and_slope(z[:, :F], case["act"])[0]
        if N != F:
            y = y * z[:, F:]
        if s.get("res") is not None:
            y = y + s["res"].to(d)
        out = [y]
        if op == "train":
            # What the checkpoint holds is defined to the bit: codes rne(fl(z / s)) of
            # fp32 values z = fl(fl(fl(fl(sum) sx) sw) + bias), s = fl(max / 127).
            w = torch.matmul(s["qx"].to(d), s["qw"].to(d).t()).to(torch.float32)
            w.mul_(s["sx"].unsqueeze(1)).mul_(s["sw"])
            if s["bias"] is not None:
                w.add_(s["bias"])
            b = _in_blocks(w, F)
            step = (b.abs().max(3, keepdim=True).values.to(d) / 127).to(torch.float32)
            b = torch.round(torch.div(b, torch.where(step > 0, step, 1))).to(d) * step.to(d)
            z = b.reshape(b.shape[0], b.shape[1], -1)[:, :, :F].reshape(z.shape)
    if op in ("act_bwd", "train"):
        value, slope = _value_and_slope(z[:, :F], case["act"])
        dy = s["dy"].to(d)
        dz = dy * slope if N == F else torch.cat([dy * slope * z[:, F:], dy * value], 1)
        out += [dz, (dz.abs() * s["sw"].to(d)).max(1).values / 127,
                (dz.abs() * s["sx"].to(d).unsqueeze(1)).max(0).values / 127, dz.sum(0)]
    return out
