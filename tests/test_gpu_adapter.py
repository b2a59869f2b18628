"""Low-rank adapters beside the shared projection, forward and backward, against
the formulas in 64 bits.

Bounds: an fp32 operand kept to 2^-17 or better (two bf16 terms; the kernels use
three), a product of two such to 2^-15 with the dropped lo lo; a sum of n terms is
within n 2^-24 of the terms' magnitudes.  The magnitudes go through the same
products with absolute values."""
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SPLIT = 2.0 ** -15


def _case(torch, M, N, K, L, R, w="bf16", dy="f32", seed=0, ids=None, runs=None):
    g = torch.Generator().manual_seed(seed)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    c = {}
    c["qx"] = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    c["qw"] = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    c["sx"] = torch.rand(M, generator=g) * 0.02 + 0.01
    c["sw"] = torch.rand(N, generator=g) * 1e-3 + 1e-4
    c["a"] = (torch.randn((L, R, K), generator=g) * K ** -0.5).to(kind[w])
    c["b"] = (torch.randn((L, N, R), generator=g) * 0.1).to(kind[w])
    c["scale"] = torch.rand(L, generator=g) + 0.5
    c["bias"] = torch.randn(N, generator=g)
    if ids is None:
        if runs:        # contiguous requests
            cuts = torch.sort(torch.randint(0, M + 1, (runs - 1,), generator=g)).values.tolist()
            ids = torch.empty(M, dtype=torch.int32)
            for a, b in zip([0] + cuts, cuts + [M]):
                ids[a:b] = int(torch.randint(-1, L, (1,), generator=g))
        else:           # any order, some without an adapter
            ids = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    c["ids"] = torch.as_tensor(ids, dtype=torch.int32)
    c["dy"] = (torch.randn((M, N), generator=g) * 0.01).to(kind[dy])
    c["qg"] = torch.randint(-127, 128, (M, N), generator=g, dtype=torch.int8)
    c["sg"] = torch.rand(M, generator=g) * 1e-4
    return c


def _cuda(c):
    return {k: v.cuda() for k, v in c.items()}


def _per_token(torch, c, key):
    """[M, ...] in 64 bits: each token's adapter's matrix; zeros without one."""
    L = c["scale"].shape[0]
    ok = (c["ids"] >= 0) & (c["ids"] < L)
    t = c[key].double()[c["ids"].clamp(0, L - 1).long()]
    return t * ok.view(-1, *[1] * (t.dim() - 1))


def _forward64(torch, c):
    x = c["qx"].double() * c["sx"].double()[:, None]
    a, b, sc = (_per_token(torch, c, k) for k in ("a", "b", "scale"))
    u = torch.bmm(a, x[:, :, None])[:, :, 0] * sc[:, None]
    usize = torch.bmm(a.abs(), x.abs()[:, :, None])[:, :, 0] * sc[:, None]
    base = (x @ c["qw"].double().T) * c["sw"].double()
    bsize = base.abs() + c["bias"].double().abs()
    y = base + c["bias"].double() + torch.bmm(b, u[:, :, None])[:, :, 0]
    ysize = torch.bmm(b.abs(), usize[:, :, None])[:, :, 0]
    return u, usize, y, bsize, ysize


def _run_fwd(qlin, d, **kw):
    return qlin.qlin_adapter_fwd(d["qx"], d["sx"], d["qw"], d["sw"], d["a"], d["b"], d["scale"],
                                 d["ids"], bias=d["bias"], **kw)


FWD = [(1, 16, 16, 1, 8), (1, 4096, 4096, 12, 16), (7, 4096, 4096, 12, 16), (16, 272, 48, 3, 24),
       (15, 64, 160, 2, 128), (17, 512, 1040, 5, 64), (33, 1040, 512, 40, 8), (130, 272, 528, 3, 40),
       (300, 528, 272, 1, 32), (611, 1024, 2048, 8, 32), (1300, 784, 400, 2, 16),
       (2500, 512, 512, 3, 16), (70, 8208, 256, 70, 16)]


@pytest.mark.parametrize("M,N,K,L,R", FWD)
@pytest.mark.parametrize("w", ["f32", "bf16"])
@pytest.mark.parametrize("runs", [None, 4])
def test_forward(M, N, K, L, R, w, runs):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    if M * N * R > 3e8 and runs is None:
        pytest.skip("the 64-bit reference holds every token's matrices")
    announce("adapter_fwd", M, N, K, L, R, w, runs)
    c = _case(torch, M, N, K, L, R, w, seed=M + R, runs=runs)
    d = _cuda(c)
    y, u = _run_fwd(qlin, d)
    y2, u2 = _run_fwd(qlin, d)
    assert torch.equal(y, y2) and torch.equal(u, u2)
    for at in range(0, M, 200):         # the reference in pieces: it holds a matrix per token
        part = {k: (v[at:at + 200] if k in ("qx", "sx", "ids") else v) for k, v in c.items()}
        u64, usize, y64, bsize, ysize = _forward64(torch, part)
        n = u64.shape[0]
        ubound = usize * (SPLIT + (K + 32) * U)
        assert ((u[at:at + n].double().cpu() - u64).abs() <= ubound).all()
        bound = 6 * U * (bsize + ysize) + ysize * (2 * SPLIT + (K + R + 64) * U)
        assert ((y[at:at + n].double().cpu() - y64).abs() <= bound).all()


def test_forward_without_adapters_is_the_projection():
    """Tokens without an adapter, or with an id outside the stack, get exactly the
    projection's values, and zeros in u."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    for M in (1, 9, 16, 40, 700):
        announce("no adapter", M)
        ids = torch.tensor([-1, 4, 1 << 30, -(1 << 31)], dtype=torch.int32).repeat(M)[:M]
        d = _cuda(_case(torch, M, 544, 256, 4, 16, ids=ids))
        y, u = _run_fwd(qlin, d)
        assert torch.equal(y, qlin.qlin_fwd(d["qx"], d["sx"], d["qw"], d["sw"], d["bias"]))
        assert (u == 0).all()


def test_forward_of_no_tokens():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    d = _cuda(_case(torch, 0, 64, 64, 2, 8))
    y, u = _run_fwd(qlin, d)
    assert y.shape == (0, 64) and u.shape == (0, 8)


@pytest.mark.parametrize("M", [5, 16, 48, 600])
def test_values_of_other_adapters_do_not_reach_a_token(M):
    """NaN and infinity in one adapter change its own tokens alone."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("isolation", M)
    c = _case(torch, M, 528, 272, 4, 16, "bf16", seed=3)
    d = _cuda(c)
    y, u = _run_fwd(qlin, d)
    d["a"][2, 3, 5] = float("nan")
    d["b"][2, 7, 1] = float("inf")
    y2, u2 = _run_fwd(qlin, d)
    other = d["ids"] != 2
    assert torch.equal(y[other], y2[other]) and torch.equal(u[other], u2[other])
    if (~other).any():
        assert u2[~other].isnan().any()


def _run_bwd(qlin, d, L, had=0, **kw):
    order, start = qlin.qlin_adapter_group(d["ids"], L)
    return qlin.qlin_adapter_bwd(d["dy"], d["qg"], d["sg"], d["qw"], d["qx"], d["sx"], d["u"],
                                 d["a"], d["b"], d["scale"], d["ids"], order, start,
                                 had_block=had, **kw)


def _rotate(torch, t, had):
    if not had:
        return t
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < had:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return (t.reshape(-1, had) @ h).reshape(t.shape) * had ** -0.5


def _rotated_size(torch, t, had):
    if not had:
        return t
    s = t.reshape(-1, had).sum(1, keepdim=True).expand(-1, had)
    return s.reshape(t.shape) * had ** -0.5


BWD = [(1, 16, 16, 1, 8, 0), (1, 512, 512, 3, 16, 128), (5, 64, 48, 2, 24, 16), (16, 272, 128, 3, 128, 64),
       (17, 144, 272, 4, 40, 0), (33, 1040, 512, 40, 8, 512), (333, 512, 512, 5, 64, 64),
       (700, 528, 1024, 2, 16, 256), (1300, 784, 384, 3, 16, 128), (2100, 256, 256, 1, 32, 32)]


@pytest.mark.parametrize("M,N,K,L,R,had", BWD)
@pytest.mark.parametrize("w,dy", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_backward(M, N, K, L, R, had, w, dy):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("adapter_bwd", M, N, K, L, R, had, w, dy)
    c = _case(torch, M, N, K, L, R, w, dy, seed=M + L, runs=5 if M > 300 else None)
    c["u"] = torch.randn((M, R), generator=torch.Generator().manual_seed(1))
    d = _cuda(c)
    dx, da, db = _run_bwd(qlin, d, L, had)
    x = c["qx"].double() * c["sx"].double()[:, None]
    D, u = c["dy"].double(), c["u"].double()
    v, vs = torch.zeros(M, R, dtype=torch.float64), torch.zeros(M, R, dtype=torch.float64)
    dx64 = (c["qg"].double() @ c["qw"].double()) * c["sg"].double()[:, None]
    base, low = dx64.abs(), torch.zeros_like(dx64)
    for l in range(L):
        at = torch.nonzero(c["ids"] == l)[:, 0]
        A, B, sc = c["a"][l].double(), c["b"][l].double(), c["scale"][l].double()
        v[at], vs[at] = sc * (D[at] @ B), sc * (D[at].abs() @ B.abs())
        dx64[at] += v[at] @ A
        low[at] += vs[at] @ A.abs()
        n = at.numel()
        want, size = v[at].T @ x[at], vs[at].T @ x[at].abs()
        got = da[l].double().cpu()
        assert ((got - want).abs() <= size * (2 * SPLIT + (N + n + 64) * U)).all()
        want, size = D[at].T @ u[at], D[at].abs().T @ u[at].abs()
        got = db[l].double().cpu()
        assert ((got - want).abs() <= size * (SPLIT + (n + 64) * U)).all()
    bound = _rotated_size(torch, base + low, had) * 16 * U
    bound = bound + _rotated_size(torch, low, had) * (2 * SPLIT + (N + R + 64) * U)
    assert ((dx.double().cpu() - _rotate(torch, dx64, had)).abs() <= bound).all()
    again = _run_bwd(qlin, d, L, had)
    for a, b in zip((dx, da, db), again):
        assert torch.equal(a, b)
    none, da2, db2 = _run_bwd(qlin, d, L, had, want_dx=False)
    assert none is None and torch.equal(da, da2) and torch.equal(db, db2)


def test_backward_of_adapters_without_tokens():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    for M in (0, 3, 40):
        announce("without tokens", M)
        c = _case(torch, M, 64, 96, 5, 16, ids=torch.full((M,), 3, dtype=torch.int32))
        c["u"] = torch.randn((M, 16))
        d = _cuda(c)
        big = torch.full((5, 16, 96), 7.0, device="cuda")
        dx, da, db = _run_bwd(qlin, d, 5, da=big)
        for l in (0, 1, 2, 4):
            assert (da[l] == 0).all() and (db[l] == 0).all()
        assert M == 0 or ((da[3] != 0).any() and (db[3] != 0).any())
        assert dx.shape == (M, 96)


def test_backward_isolation():
    """A NaN in one token's row reaches its own adapter's gradients alone."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    c = _case(torch, 90, 80, 96, 3, 16, seed=4)
    c["u"] = torch.randn((90, 16))
    d = _cuda(c)
    dx, da, db = _run_bwd(qlin, d, 3)
    t = int(torch.nonzero(c["ids"] == 1)[0, 0])
    d["dy"][t, 3] = float("nan")
    d["a"][1, 0, 0] = float("inf")
    dx2, da2, db2 = _run_bwd(qlin, d, 3)
    for l in (0, 2):
        assert torch.equal(da[l], da2[l]) and torch.equal(db[l], db2[l])
    other = d["ids"] != 1
    assert torch.equal(dx[other], dx2[other])
    assert da2[1].isnan().any() and db2[1].isnan().any()


def test_gradients_against_differences():
    """sum(dY * y) is linear in A, B and x^ one at a time: its central differences
    in 64 bits are exact to their rounding."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K, L, R = 50, 96, 64, 3, 16
    c = _case(torch, M, N, K, L, R, "f32", "f32", seed=8)
    # A gradient that its INT8 codes hold exactly: dY sw = sg qg.
    c["sw"] = torch.full((N,), 2.0 ** -10)
    c["sg"] = torch.full((M,), 2.0 ** -14)
    c["dy"] = c["qg"].float() * 2.0 ** -4
    d = _cuda(c)
    _, d["u"] = _run_fwd(qlin, d)
    dx, da, db = _run_bwd(qlin, d, L)
    x0 = c["qx"].double() * c["sx"].double()[:, None]

    def loss(x, a, b):
        sc = _per_token(torch, c, "scale")
        A = _per_token(torch, {**c, "a": a}, "a")
        B = _per_token(torch, {**c, "b": b}, "b")
        u = torch.bmm(A, x[:, :, None]) * sc[:, None, None]
        y = (x @ c["qw"].double().T) * c["sw"].double() + torch.bmm(B, u)[:, :, 0]
        return (c["dy"].double() * y).sum()

    g = torch.Generator().manual_seed(2)
    a0, b0 = c["a"].double(), c["b"].double()
    for name, got, at in (("x", dx, x0), ("a", da, a0), ("b", db, b0)):
        for _ in range(3):
            t = torch.randn(at.shape, generator=g, dtype=torch.float64)
            args = lambda s: dict(x=x0, a=a0, b=b0) | {name: at + s * t}       # noqa: E731
            diff = (loss(**args(0.5)) - loss(**args(-0.5)))
            inner = got.double().cpu() * t
            bound = inner.abs().sum() * (4 * SPLIT + (N + M + K) * U) * 4
            assert abs(diff - inner.sum()) <= bound, name


@pytest.mark.parametrize("M,L", [(0, 1), (1, 1), (63, 2), (64, 7), (1000, 1023), (5000, 3), (777, 40)])
def test_group(M, L):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("adapter_group", M, L)
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-2, L + 2, (M,), generator=g, dtype=torch.int32)
    order, start = qlin.qlin_adapter_group(ids.cuda(), L)
    key = torch.where((ids >= 0) & (ids < L), ids, L)
    assert torch.equal(order.cpu(), torch.sort(key, stable=True).indices.to(torch.int32))
    want = torch.searchsorted(torch.sort(key).values, torch.arange(L + 1, dtype=torch.int32))
    assert torch.equal(start.cpu(), want.to(torch.int32))


def test_other_stream_and_graph():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K, L, R = 400, 512, 2048, 3, 16
    d = _cuda(_case(torch, M, N, K, L, R, "bf16", "bf16", seed=1, runs=4))
    wf = torch.zeros(qlin.qlin_adapter_fwd_ws_bytes(M, N, K, L, R), dtype=torch.uint8, device="cuda")
    wb = torch.zeros(qlin.qlin_adapter_bwd_ws_bytes(M, N, K, L, R), dtype=torch.uint8, device="cuda")

    def both():
        y, d["u"] = _run_fwd(qlin, d, workspace=wf)
        return [y, d["u"], *_run_bwd(qlin, d, L, 128, workspace=wb)]

    want = [t.clone() for t in both()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(3):
        d["dy"].copy_(torch.randn((M, N), device="cuda") * 0.01)
        want = [t.clone() for t in both()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)


def test_one_workspace_for_all_calls():
    """Forward and backward calls of different shapes, one after another on one
    workspace, give what fresh ones give, whole and split contractions alike."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    shapes = [(40, 512, 2048, 3, 16, "bf16"), (700, 2304, 1024, 2, 64, "f32"), (5, 64, 512, 2, 8, "f32"),
              (40, 4096, 512, 4, 128, "f32"), (1500, 2304, 2304, 3, 24, "bf16"), (33, 512, 2048, 3, 16, "bf16")]
    size = max(max(qlin.qlin_adapter_fwd_ws_bytes(*s[:5]), qlin.qlin_adapter_bwd_ws_bytes(*s[:5]))
               for s in shapes)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for k, (M, N, K, L, R, w) in enumerate(shapes * 2):
        announce("shared workspace", M, N, K, L, R, w)
        d = _cuda(_case(torch, M, N, K, L, R, w, "bf16", seed=k, runs=3))
        got = [*_run_fwd(qlin, d, workspace=ws)]
        d["u"] = got[1]
        got += _run_bwd(qlin, d, L, 128, workspace=ws)
        want = [*_run_fwd(qlin, d)] + [*_run_bwd(qlin, d, L, 128)]
        for a, b in zip(want, got):
            assert torch.equal(a, b)
