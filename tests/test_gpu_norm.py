"""The RMS norm with INT8 rows as its output, and its backward, against the
formulas in 64 bits.  Bounds are the rounding errors' own: a sum of n fp32 terms
in the kernel's order (at most CHAIN additions one after another) is within
CHAIN 2^-24 of the sum of the terms' magnitudes, a product or sum within 2^-24."""
import math

import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


def _chain(cols):
    """Additions behind one another in a row's sum: a lane's own elements, then
    the lanes and waves."""
    return 8 * 16 + 6 + 16 if cols > 16384 else 8 * 16 + 6 + 4


def _hadamard(torch, n):
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h / math.sqrt(n)


def _rows(torch, rows, cols, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * std
    x[:, ::37] *= 8
    if rows > 2:
        x[rows // 2] = 0
    return x.to(dtype).cuda()


def _forward64(torch, h, gamma, had):
    """n, rotated values and the bound of the kernel's error in them."""
    h = h.double().cpu()
    gamma = gamma.double().cpu()
    rstd = 1 / torch.sqrt(h.square().mean(1) + EPS)
    n = h * rstd[:, None] * gamma
    rel = (_chain(h.shape[1]) / 2 + 4) * U + 2 * U          # rstd's, then two products
    if not had:
        return rstd, n, n.abs() * rel
    k = had
    rot = (n.view(-1, k) @ _hadamard(torch, k)).view(n.shape)
    size = n.abs().view(-1, k).sum(1, keepdim=True).expand(-1, k).reshape(n.shape) / math.sqrt(k)
    return rstd, rot, size * (rel + (math.log2(k) + 2) * U)


SHAPES = [(1, 16, 0), (1, 16, 16), (3, 4096, 128), (5, 48, 16), (7, 2064, 0), (2, 2048, 512),
          (257, 640, 128), (33, 5376, 128), (2, 8192, 64), (3, 16384, 2), (2, 16400, 16),
          (2, 40960, 128), (1, 131072, 256), (1, 70000, 0), (1100, 4096, 128), (2500, 1808, 16)]


@pytest.mark.parametrize("rows,cols,had", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [True, False])
def test_forward(rows, cols, had, dtype, residual):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("rmsnorm_quant", rows, cols, had, dtype, residual)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = _rows(torch, rows, cols, dt, 1)
    res = _rows(torch, rows, cols, dt, 2, 2.0) if residual else None
    gamma = (1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).cuda()
    q, s, h, rstd, y = qlin.qlin_rmsnorm_quant(x, gamma, EPS, residual=res, had_block=had,
                                               want_y=True)
    if residual:
        assert torch.equal(h, (x.float() + res.float()).to(dt))
    else:
        assert h is x
    r64, g64, err = _forward64(torch, h, gamma, had)
    assert ((rstd.double().cpu() - r64).abs() <= r64 * (_chain(cols) / 2 + 4) * U).all()
    s64 = s.double().cpu()
    amax = g64.abs().amax(1)
    slack = err.amax(1)
    assert ((s64 * 127 - amax).abs() <= slack + 4 * U * amax).all()
    # The code is the nearest integer to a quotient whose error is err / s.
    off = (q.double().cpu() * s64[:, None] - g64).abs()
    assert (off <= s64[:, None] * (0.5 + 2.0 ** -16) + err).all()
    assert (q.to(torch.int16).abs() <= 127).all()
    assert (q[s == 0] == 0).all()
    assert torch.equal(y, (q.float() * s[:, None]).to(torch.bfloat16))


def test_forward_matches_the_quantizer_bit_for_bit():
    """With gamma 1 the rounded normalized row goes through the same quantizer as
    qlin_quantize_rows, rotation included."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    x = _rows(torch, 40, 2048, torch.float32, 5)
    gamma = torch.ones(2048, device="cuda")
    for had in (0, 32, 64, 128):
        announce("rmsnorm_quant against quantize_rows", had)
        q, s, _, rstd, _ = qlin.qlin_rmsnorm_quant(x, gamma, EPS, had_block=had)
        q2, s2 = qlin.qlin_quantize_rows(x * rstd[:, None], had_block=had)
        assert torch.equal(q, q2) and torch.equal(s, s2)


def test_in_place_and_other_stream():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    x, r = _rows(torch, 65, 1024, torch.bfloat16, 1), _rows(torch, 65, 1024, torch.bfloat16, 2)
    gamma = torch.ones(1024, device="cuda")
    want = qlin.qlin_rmsnorm_quant(x, gamma, EPS, residual=r, had_block=128, want_y=True)
    r2 = r.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = qlin.qlin_rmsnorm_quant(x, gamma, EPS, residual=r2, h=r2, had_block=128, want_y=True,
                                  stream=side)
    side.synchronize()
    assert got[2] is r2
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_rows_that_are_not_finite():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    for cols, value, at in ((512, float("nan"), 7), (512, float("inf"), 0), (4096, -float("inf"), 9),
                            (40960, float("nan"), 5), (512, 3e38, 1)):
        announce("not finite", cols, value)
        x = _rows(torch, 9, cols, torch.float32, 1)
        clean = qlin.qlin_rmsnorm_quant(x, torch.ones(cols, device="cuda"), EPS, had_block=128)
        x[4, at] = value        # 3e38: its square overflows
        q, s, _, rstd, y = qlin.qlin_rmsnorm_quant(x, torch.ones(cols, device="cuda"), EPS,
                                                   had_block=128, want_y=True)
        assert s[4].isnan() and (q[4] == 0).all() and y[4].isnan().all()
        keep = torch.arange(9, device="cuda") != 4
        assert torch.equal(q[keep], clean[0][keep]) and torch.equal(s[keep], clean[1][keep])
    gamma = torch.ones(512, device="cuda")
    gamma[3] = float("nan")
    _, s, _, _, _ = qlin.qlin_rmsnorm_quant(_rows(torch, 2, 512, torch.float32, 1), gamma, EPS)
    assert s.isnan().all()


def test_tiny_rows():
    """Rows so small that eps alone is under the root, down to scales below the
    normal range."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    for scale in (1e-20, 1e-36, 1e-40, 1e-44):
        announce("tiny", scale)
        x = _rows(torch, 4, 256, torch.float32, 1) * scale
        gamma = torch.full((256,), 1e-3, device="cuda")
        q, s, _, rstd, _ = qlin.qlin_rmsnorm_quant(x, gamma, EPS)
        n = (x * rstd[:, None]) * gamma
        a = n.abs().amax(1)
        want = a / 127.0
        assert torch.equal(s, want)
        code = torch.where(want[:, None] > 0, n / want[:, None], 0.0).round().clamp(-127, 127)
        assert torch.equal(q.float(), code)


BWD = [(1, 16), (1, 4096), (2, 48), (7, 2064), (300, 640), (33, 5376), (1700, 1024), (3, 8192),
       (5, 8208), (2, 40960), (130, 16384)]


@pytest.mark.parametrize("rows,cols", BWD)
@pytest.mark.parametrize("dtype,dn_dtype,with_res", [("f32", "f32", True), ("bf16", "f32", True),
                                                     ("bf16", "bf16", False), ("f32", "bf16", False)])
def test_backward(rows, cols, dtype, dn_dtype, with_res):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("rmsnorm_bwd", rows, cols, dtype, dn_dtype, with_res)
    kinds = {"f32": torch.float32, "bf16": torch.bfloat16}
    h = _rows(torch, rows, cols, kinds[dtype], 1, 2.0)
    dn = _rows(torch, rows, cols, kinds[dn_dtype], 2, 0.01)
    dres = _rows(torch, rows, cols, kinds[dtype], 3, 0.01) if with_res else None
    gamma = (1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(4))).cuda()
    rstd = (1 / torch.sqrt(h.float().square().mean(1) + EPS))
    dh, dgamma = qlin.qlin_rmsnorm_bwd(dn, h, rstd, gamma, dres=dres)
    H, D, R, G = (t.double().cpu() for t in (h, dn, rstd, gamma))
    xh = H * R[:, None]
    g = D * G
    dot = (g * xh).mean(1, keepdim=True)
    want = R[:, None] * (g - xh * dot)
    size = R[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if with_res:
        want = want + dres.double().cpu()
        size = size + dres.double().cpu().abs()
    chain = max(_chain(cols), 8 * -(-cols // 8192) + 6 + 16)
    bound = size * (chain + 8) * U + (want.abs() * 2.0 ** -8 if dtype == "bf16" else 0)
    assert ((dh.double().cpu() - want).abs() <= bound).all()
    want = (D * xh).sum(0)
    size = (D * xh).abs().sum(0)
    # rows of one workgroup, then 16 lanes of partial sums: at most all of them
    bound = size * (min(rows, -(-rows // 64) + 64 + 16) + 4) * U
    assert ((dgamma.double().cpu() - want).abs() <= bound).all()
    dh2, dgamma2 = qlin.qlin_rmsnorm_bwd(dn, h, rstd, gamma, dres=dres)
    assert torch.equal(dh, dh2) and torch.equal(dgamma, dgamma2)


def test_backward_of_no_rows():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    e = torch.empty((0, 64), device="cuda")
    dh, dgamma = qlin.qlin_rmsnorm_bwd(e, e, torch.empty(0, device="cuda"),
                                       torch.ones(64, device="cuda"))
    assert dh.shape == (0, 64) and (dgamma == 0).all()
    q, s, _, _, _ = qlin.qlin_rmsnorm_quant(e, torch.ones(64, device="cuda"), EPS)
    assert q.shape == (0, 64) and s.shape == (0,)


def test_backward_against_differences():
    """Along random directions, central differences of sum(dn * n) in 64 bits."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    gen = torch.Generator().manual_seed(9)
    h = torch.randn((6, 320), generator=gen, dtype=torch.float32)
    dn = torch.randn((6, 320), generator=gen, dtype=torch.float32)
    gamma = torch.rand(320, generator=gen) + 0.5

    def loss(h, gamma):
        rstd = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        return (dn.double() * h * rstd * gamma).sum()

    rstd = 1 / torch.sqrt(h.square().mean(1) + EPS)
    dh, dgamma = qlin.qlin_rmsnorm_bwd(dn.cuda(), h.cuda(), rstd.cuda(), gamma.cuda())
    H, G, step = h.double(), gamma.double(), 1e-5
    for k in range(4):
        d = torch.randn(h.shape, generator=gen, dtype=torch.float64)
        diff = (loss(H + step * d, G) - loss(H - step * d, G)) / (2 * step)
        got = (dh.double().cpu() * d).sum()
        # differences: step^2 times a third derivative of order one, 1e-16 / step
        # of the loss; the kernel's: 2^-18 of the terms
        assert abs(diff - got) <= (1e-6 + 2.0 ** -18) * (dh.double().cpu() * d).abs().sum()
        d = torch.randn(320, generator=gen, dtype=torch.float64)
        diff = (loss(H, G + step * d) - loss(H, G - step * d)) / (2 * step)
        got = (dgamma.double().cpu() * d).sum()
        assert abs(diff - got) <= (1e-6 + 2.0 ** -18) * (dgamma.double().cpu() * d).abs().sum()


def test_graph_replay():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    x, r = _rows(torch, 70, 1024, torch.bfloat16, 1), _rows(torch, 70, 1024, torch.bfloat16, 2)
    gamma = torch.ones(1024, device="cuda")
    dn = _rows(torch, 70, 1024, torch.float32, 3)
    ws = torch.empty(qlin.qlin_rmsnorm_bwd_ws_bytes(70, 1024), dtype=torch.uint8, device="cuda")

    def both():
        q, s, h, rstd, y = qlin.qlin_rmsnorm_quant(x, gamma, EPS, residual=r, had_block=128,
                                                   want_y=True)
        return [q, s, h, rstd, y, *qlin.qlin_rmsnorm_bwd(dn, h, rstd, gamma, workspace=ws)]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(3):
        x.copy_(_rows(torch, 70, 1024, torch.bfloat16, 10 + k))
        want = [t.clone() for t in both()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)
