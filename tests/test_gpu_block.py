"""The operators inside a feed-forward block against the formulas in 64 bits
(block_ref has the bounds).  The sums before the activation are qlin_fwd's to the bit,
so everything after them is compared from those."""
import pytest

from tests import block_ref as ref
from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
U = ref.U


def _dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _operands(torch, M, N, K, seed=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    qx = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    qw = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    sx = torch.rand(M, generator=g) + 0.5
    sw = (torch.rand(N, generator=g) + 0.5) * (2.0 / (K ** 0.5 * 73 * 73))
    if M > 4:
        sx[M // 2] = 0                  # an empty row: z is the bias
        qx[M // 2] = 0
        sx[1] *= 40                     # a large one: saturated activations
    b = torch.randn(N, generator=g) if bias else None
    return [None if t is None else t.cuda() for t in (qx, sx, qw, sw, b)]


def _near(torch, got, want, err, what):
    got, step = got.cpu(), ref.STEP[got.dtype]
    off = (got.double() - want).abs()
    room = err + (want.abs() + err) * step + U * want.abs()
    bad = ~(off <= room)
    assert not bad.any(), (what, int(bad.sum()), float((off / room.clamp(min=1e-300)).max()))


def _guarded(torch, shape, dtype):
    """An output between rows of a pattern, and a check that they are whole."""
    pad = 4096
    n = shape[0] * shape[1]
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n * size + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    out = raw[pad:pad + n * size].view(dtype).view(shape)

    def whole():
        assert (raw[:pad] == 0x5A).all() and (raw[pad + n * size:] == 0x5A).all()
    return out, whole


SHAPES = [(1, 16, 16), (1, 4096, 256), (3, 48, 80), (16, 272, 4096), (16, 32, 1040), (5, 48, 2064), (9, 6416, 528),
          (12, 6432, 1040), (4, 4096, 3088), (8, 4112, 1008), (17, 16, 16),
          (33, 144, 1168), (255, 528, 64), (257, 1040, 192), (300, 2064, 400), (1000, 784, 256)]
# The tiles of few tokens, each size: 32, 64 and 128 tokens per workgroup, four and eight
# waves; and calls just past them, of 256 x 256 tiles.
SHAPES += [(32, 80, 528), (64, 6416, 272), (50, 8240, 80), (65, 48, 1040), (100, 6416, 528), (129, 6416, 48),
           (161, 10944, 64), (513, 4112, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_act_forward(M, N, K, act):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    qx, sx, qw, sw, b = _operands(torch, M, N, K)
    z = qlin.qlin_fwd(qx, sx, qw, sw, bias=b)
    g = torch.Generator().manual_seed(9)
    for y_type, r_type in (("f32", None), ("bf16", None), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"),
                           ("f32", "f32")):
        announce("fwd_act", M, N, K, act, y_type, r_type)
        res = None if r_type is None else (3 * torch.randn((M, N), generator=g)).to(_dt(torch, r_type)).cuda()
        y, whole = _guarded(torch, (M, N), _dt(torch, y_type))
        want, err = ref.forward(z.cpu(), N, act, None if res is None else res.cpu())
        out = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, act=act, residual=res, y=y)
        assert out[0] is y and out[1] is None and out[2] is None
        whole()
        _near(torch, y, want, err, (y_type, r_type))
        ck, whole_ck = _guarded(torch, (M, N), torch.int8)
        again, c, s = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, act=act, residual=res,
                                        dtype=_dt(torch, y_type), ck=ck, save=True)
        whole_ck()
        assert torch.equal(again, y)            # (the tile kernel and the streaming one agree)
        codes, scales = ref.checkpoint(z.cpu(), N)
        assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu(), codes)
        if act == "none" and res is None:
            assert torch.equal(y, z.to(y.dtype))


@pytest.mark.parametrize("M,F,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_gated_forward(M, F, K, act):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    for bias, y_type in ((True, "f32"), (False, "bf16")):
        announce("fwd_gated", M, F, K, act, bias, y_type)
        qx, sx, qw, sw, b = _operands(torch, M, 2 * F, K, 1, bias)
        z = qlin.qlin_fwd(qx, sx, qw, sw, bias=b).cpu()
        y, whole = _guarded(torch, (M, F), _dt(torch, y_type))
        want, err = ref.forward(z, F, act)
        qlin.qlin_fwd_gated(qx, sx, qw, sw, bias=b, act=act, y=y)
        whole()
        _near(torch, y, want, err, y_type)
        ck, whole_ck = _guarded(torch, (M, 2 * F), torch.int8)
        again, c, s = qlin.qlin_fwd_gated(qx, sx, qw, sw, bias=b, act=act, dtype=y.dtype, ck=ck, save=True)
        whole_ck()
        assert torch.equal(again, y)
        codes, scales = ref.checkpoint(z, F)
        assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu(), codes)


@pytest.mark.parametrize("M,N,K", [(1000, 8480, 1040), (611, 14336, 1024), (600, 8160, 4112), (700, 2816, 1552),
                                   (1300, 11744, 1552)])
def test_many_tiles(M, N, K):
    """Whole tiles, and last rounds of tiles that are split along the contraction in two
    and three; one workspace that both calls and the plain product use in turn."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    qx, sx, qw, sw, b = _operands(torch, M, N, K, 3)
    ws = torch.zeros(max(qlin.qlin_fwd_act_ws_bytes(M, N, K), qlin.qlin_fwd_gated_ws_bytes(M, N // 2, K),
                         qlin.qlin_product_ws_bytes(0, M, N, K)), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        announce("split tiles", M, N, K)
        z = qlin.qlin_product_ws(0, qx, sx, qw, M, N, K, scol=sw, bias=b, workspace=ws)
        y, c, s = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, dtype=torch.float32, save=True, workspace=ws)
        assert torch.equal(y, z)
        codes, scales = ref.checkpoint(z.cpu(), N)
        assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu(), codes)
        F = N // 2
        y, c, s = qlin.qlin_fwd_gated(qx, sx, qw, sw, bias=b, dtype=torch.float32, save=True, workspace=ws)
        want, err = ref.forward(z.cpu(), F, "silu")
        _near(torch, y, want, err, "gated")
        codes, scales = ref.checkpoint(z.cpu(), F)
        assert torch.equal(s.cpu(), scales) and torch.equal(c.cpu(), codes)


def _checkpointed(torch, M, F, gated, seed):
    g = torch.Generator().manual_seed(seed)
    z = 2 * torch.randn((M, 2 * F if gated else F), generator=g)
    z[:, ::53] *= 6
    if M > 3:
        z[2] = 0
    return ref.checkpoint(z, F)


BACK = [(1, 16), (1, 4096), (2, 48), (15, 528), (16, 512), (17, 1040), (100, 80), (333, 1808), (1025, 272),
        (2000, 1024), (37, 14336)]


@pytest.mark.parametrize("M,F", BACK)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_backward(M, F, act, gated):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    N = 2 * F if gated else F
    ck, ck_s = _checkpointed(torch, M, F, gated, 5)
    g = torch.Generator().manual_seed(6)
    sw, sx = torch.rand(N, generator=g) + 0.1, torch.rand(M, generator=g) + 0.1
    for dy_type, dz_type in (("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")):
        announce("act_bwd", M, F, act, gated, dy_type, dz_type)
        dy = torch.randn((M, F), generator=g).to(_dt(torch, dy_type))
        if M > 6:
            dy[5] = 0
        want, err = ref.backward(dy, ref.restored(ck, ck_s, F), F, act)
        dz, whole = _guarded(torch, (M, N), _dt(torch, dz_type))
        out, s1, s2, db = qlin.qlin_act_bwd(dy.cuda(), ck.cuda(), ck_s.cuda(), act, gated=gated, sw=sw.cuda(),
                                            sx=sx.cuda(), dz=dz, want_db=True)
        assert out is dz
        whole()
        _near(torch, dz, want, err, "dz")
        for got, scale, over in ((s1, sw, 1), (s2, sx[:, None], 0)):
            m = (want * scale).abs().amax(over)
            room = (err * scale).amax(over) + 4 * U * m     # (a product, a quotient)
            assert ((got.double().cpu() * 127 - m).abs() <= room).all()
        # At most M additions one after another.
        room = err.sum(0) + M * U * want.abs().sum(0)
        assert ((db.double().cpu() - want.sum(0)).abs() <= room).all()
        if M > 6:
            assert (dz[5] == 0).all() and s1[5] == 0
        again = qlin.qlin_act_bwd(dy.cuda(), ck.cuda(), ck_s.cuda(), act, gated=gated, dtype=dz.dtype)
        assert torch.equal(again[0], dz) and again[1:] == (None, None, None)


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """dz is the derivative of sum(dy y) by z: central differences of the formula in
    64 bits, whose own error at h = 2^-16 is below h^2 (third derivative below 6 here)
    plus 2^-52 / h of the terms."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("act_bwd against differences", act)
    M, F, h = 12, 64, 2.0 ** -16
    for gated in (False, True):
        ck, ck_s = _checkpointed(torch, M, F, gated, 8)
        z = ref.restored(ck, ck_s, F)
        dy = torch.randn((M, F), generator=torch.Generator().manual_seed(3))
        dz = qlin.qlin_act_bwd(dy.cuda(), ck.cuda(), ck_s.cuda(), act, gated=gated, dtype=torch.float32)[0]

        def f(zz):
            v = ref.act(zz[:, :F], act)[0]
            return dy.double() * (v * zz[:, F:] if gated else v)

        for half in range(2 if gated else 1):
            at = slice(half * F, (half + 1) * F)
            up, down = z.double(), z.double()
            up[:, at] += h
            down[:, at] -= h
            diff = (f(up) - f(down)) / (2 * h)
            _, err = ref.backward(dy, z, F, act)
            u = z[:, F:].double().abs() if gated else torch.ones(M, F, dtype=torch.float64)
            room = err[:, at] + (dy.abs().double() * (1 + u) * (1 + z.double().abs().amax()) * (h * h + 2.0 ** -36)
                                 + U * diff.abs())
            clear = z[:, :F].abs() > 2 * h if act == "relu" else torch.ones(M, F, dtype=torch.bool)
            off = (dz[:, at].double().cpu() - diff).abs()
            assert (off <= room)[clear].all(), float((off / room)[clear].max())


@pytest.mark.parametrize("M,N", [(1, 16), (3, 528), (16, 64), (100, 1040), (513, 2064)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_for_known_scales(M, N, dtype):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("quantize_grad_scaled", M, N, dtype)
    g = torch.Generator().manual_seed(1)
    dy = torch.randn((M, N), generator=g)
    dy[:, 3] = 0
    dy[M // 2] *= 1e-30
    dy = dy.to(_dt(torch, dtype)).cuda()
    sw, sx = (torch.rand(N, generator=g) + 0.1).cuda(), (torch.rand(M, generator=g) + 0.1).cuda()
    q1, s1, q2, s2, _ = qlin.qlin_quantize_grad(dy, sw, sx)
    got = qlin.qlin_quantize_grad_scaled(dy, sw, sx, s1, s2)
    assert torch.equal(got[0], q1) and torch.equal(got[1], q2)


@pytest.mark.parametrize("gated", [False, True])
def test_codes_of_a_rounded_gradient(gated):
    """dz in bf16 with the scales of its fp32 values: a code is the nearest integer to
    dz sw / s1 (two roundings), never past 127 in magnitude."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("act_bwd, then its codes", gated)
    M, F = 700, 784
    N = 2 * F if gated else F
    ck, ck_s = _checkpointed(torch, M, F, gated, 2)
    g = torch.Generator().manual_seed(7)
    sw, sx = (torch.rand(N, generator=g) + 0.1).cuda(), (torch.rand(M, generator=g) + 0.1).cuda()
    dy = torch.randn((M, F), generator=g).cuda()
    dz, s1, s2, _ = qlin.qlin_act_bwd(dy, ck.cuda(), ck_s.cuda(), "silu", gated=gated, sw=sw, sx=sx)
    q1, q2 = qlin.qlin_quantize_grad_scaled(dz, sw, sx, s1, s2)
    for q, v, s in ((q1, dz.double() * sw, s1[:, None]), (q2, dz.double() * sx[:, None], s2[None])):
        off = (q.double() * s - v).abs()
        assert (off <= s.double() * (0.5 + 127.5 * 3 * U)).all()
        assert int(q.to(torch.int16).abs().max()) == 127


def test_not_finite_values_stay_in_their_place():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, F, K = 40, 208, 64
    for gated in (False, True):
        announce("not finite", gated)
        N = 2 * F if gated else F
        first = qlin.qlin_fwd_gated if gated else qlin.qlin_fwd_act
        qx, sx, qw, sw, b = _operands(torch, M, N, K, 4)
        clean = first(qx, sx, qw, sw, bias=b, act="silu", dtype=torch.float32, save=True)
        sx2, b2 = sx.clone(), b.clone()
        sx2[7], sx2[8], b2[70] = float("nan"), float("inf"), float("nan")
        y, ck, ck_s = first(qx, sx2, qw, sw, bias=b2, act="silu", dtype=torch.float32, save=True)
        rows = [m for m in range(M) if m not in (7, 8)]
        cols = [n for n in range(F) if n != 70]
        assert torch.equal(y[rows][:, cols], clean[0][rows][:, cols])
        assert y[7].isnan().all() and y[:, 70].isnan().all() and not y[8].isfinite().any()
        blocks = [k for k in range(ck_s.shape[1]) if k != 2]
        assert torch.equal(ck_s[rows][:, blocks], clean[2][rows][:, blocks])
        assert not ck_s[7].isfinite().any() and not ck_s[:, 2].isfinite().any()
        dy = torch.ones((M, F), device="cuda")
        dz, s1, s2, db = qlin.qlin_act_bwd(dy, ck, ck_s, "silu", gated=gated, sw=torch.ones_like(sw),
                                           sx=torch.ones_like(sx), dtype=torch.float32, want_db=True)
        assert not s1.isfinite().any() and not s2[64:96].isfinite().any() and not db[64:96].isfinite().any()
        assert not dz[7].isfinite().any() and not dz[8].isfinite().any()
        keep = [n for n in range(F) if n // 32 != 2]
        want = qlin.qlin_act_bwd(dy, clean[1], clean[2], "silu", gated=gated, dtype=torch.float32)[0]
        assert torch.equal(dz[rows][:, keep], want[rows][:, keep])


def test_no_tokens():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("no tokens")
    qx, sx, qw, sw, b = _operands(torch, 0, 64, 32, 0)
    y, ck, ck_s = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, save=True)
    assert y.shape == (0, 64) and ck_s.shape == (0, 2)
    y, ck, ck_s = qlin.qlin_fwd_gated(qx, sx, qw, sw, bias=b, save=True)
    assert y.shape == (0, 32) and ck.shape == (0, 64)
    s2, db = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    qlin.qlin_act_bwd(y, ck, ck_s, "silu", gated=True, sw=sw, sx=sx, s2=s2, db=db)
    assert (s2 == 0).all() and (db == 0).all()


def test_residual_in_place():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    for M in (5, 700):
        for dtype in (torch.float32, torch.bfloat16):
            announce("residual in place", M, dtype)
            qx, sx, qw, sw, b = _operands(torch, M, 528, 256, 6)
            res = torch.randn((M, 528), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
            want = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, act="relu", residual=res, dtype=dtype)[0]
            got = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, act="relu", residual=res, y=res)[0]
            assert got is res and torch.equal(got, want)


def _pass(qlin, torch, ops, dy, gated, stream=None):
    first = qlin.qlin_fwd_gated if gated else qlin.qlin_fwd_act
    qx, sx, qw, sw, b = ops
    y, ck, ck_s = first(qx, sx, qw, sw, bias=b, act="gelu", save=True, stream=stream)
    dz, s1, s2, db = qlin.qlin_act_bwd(dy, ck, ck_s, "gelu", gated=gated, sw=sw, sx=sx, want_db=True,
                                       stream=stream)
    q1, q2 = qlin.qlin_quantize_grad_scaled(dz, sw, sx, s1, s2, stream=stream)
    return y, ck, ck_s, dz, s1, s2, db, q1, q2


@pytest.mark.parametrize("gated", [False, True])
def test_other_stream_and_replayed_graph(gated):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K = 520, 4608, 256
    ops = _operands(torch, M, N, K, 2)
    F = N // 2 if gated else N
    dy = torch.randn((M, F), generator=torch.Generator().manual_seed(4)).cuda()
    want = _pass(qlin, torch, ops, dy, gated)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    announce("block on another stream", gated)
    got = _pass(qlin, torch, ops, dy, gated, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    announce("block in a graph", gated)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _pass(qlin, torch, ops, dy, gated)
    other = _operands(torch, M, N, K, 12)
    for k in range(3):
        for t, v in zip(ops, other if k == 1 else _operands(torch, M, N, K, 2)):
            t.copy_(v)
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = _pass(qlin, torch, ops, dy, gated)
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), k


def test_two_graphs_share_a_workspace():
    """Replays in turn on one stream, eager calls with it between them."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K = 600, 8160, 4112
    ops = _operands(torch, M, N, K, 5)
    need = max(qlin.qlin_fwd_act_ws_bytes(M, N, K), qlin.qlin_fwd_gated_ws_bytes(M, N // 2, K))
    assert need
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    calls = [lambda: qlin.qlin_fwd_act(*ops[:4], bias=ops[4], act="gelu", workspace=ws)[0],
             lambda: qlin.qlin_fwd_gated(*ops[:4], bias=ops[4], act="silu", workspace=ws)[0]]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    announce("two graphs, one workspace")
    graphs, held = [], []
    for f in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(f())
    for k in range(4):
        for h in held:
            h.zero_()
        for g in graphs if k % 2 else graphs[::-1]:
            g.replay()
        again = calls[k % 2]()
        torch.cuda.synchronize()
        assert torch.equal(again, want[k % 2]) and all(torch.equal(h, w) for h, w in zip(held, want)), k


def test_two_streams_at_once():
    """Calls with workspaces of their own do not share anything."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("block on two streams at once")
    sets = [(_operands(torch, 300, 4608, 512, k), torch.randn((300, 2304), device="cuda")) for k in (1, 2)]
    want = [_pass(qlin, torch, o, d, True) for o, d in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [_pass(qlin, torch, o, d, True, stream=s) for (o, d), s in zip(sets, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refused_calls_leave_outputs_untouched():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("refusals")
    qx, sx, qw, sw, b = _operands(torch, 20, 64, 32, 0)
    y = torch.full((20, 64), 7.0, device="cuda")
    with pytest.raises(ValueError):
        qlin.qlin_fwd_act(qx, sx, qw, sw, act="swish", y=y)
    with pytest.raises(ValueError):
        qlin.qlin_fwd_act(qx, sx, qw, sw, y=y[:, :32])
    with pytest.raises(TypeError):
        qlin.qlin_fwd_act(qx, sx, qw, sw, y=y.half())
    with pytest.raises(ValueError):
        qlin.qlin_fwd_act(qx, sx, qw, sw.cpu(), y=y)
    with pytest.raises(qlin.QlinError):             # y over qx
        qlin.qlin_fwd_act(qx, sx, qw[:16].contiguous(), sw[:16].contiguous(),
                          y=qx.view(torch.bfloat16))
    with pytest.raises(qlin.QlinError):
        qlin.qlin_fwd_gated(qx, sx, qw[:48].contiguous(), sw[:48].contiguous(), y=y[:, :24].contiguous())
    ck, ck_s = torch.zeros((20, 64), dtype=torch.int8, device="cuda"), torch.zeros((20, 2), device="cuda")
    with pytest.raises(ValueError):
        qlin.qlin_act_bwd(y, ck, ck_s, "silu", s1=torch.zeros(20, device="cuda"))
    with pytest.raises(ValueError):
        qlin.qlin_act_bwd(y, ck, ck_s, "silu", gated=True)
    with pytest.raises(ValueError):
        qlin.qlin_act_bwd(y, ck, torch.zeros((20, 4), device="cuda"), "silu")
    assert (y == 7).all()
