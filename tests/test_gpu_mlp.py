"""The feed-forward block as a layer: its forward and backward from its own INT8
state, its updates, and several passes kept at once."""
import pytest

from tests import block_ref as ref
from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def _block(torch, M, K, F, N, gated, act, dtype, had=128, seed=0):
    import w8a8_integer_linear_amd as qlin
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (std * torch.randn(s, generator=g)).cuda()        # noqa: E731
    rows = 2 * F if gated else F
    block = qlin.MLPW8A8Training(r(rows, K, std=K ** -0.5), r(N, F, std=F ** -0.5), r(rows, std=0.1),
                                 r(N, std=0.1), act=act, gated=gated, had_block=had, dtype=dtype)
    return block, r(M, K).to(dtype), r(M, N).to(dtype), r(M, N, std=0.1)


def _product(torch, q, s, w):
    """fl(fl32(sum) s) in 64 bits from INT8 operands [M, T] and [T, N]."""
    return (q.double().cpu() @ w.double().cpu()) * s.double().cpu()[:, None]


CASES = [(1, 256, 384, 256, True, "silu", "bf16", 128), (33, 128, 272, 128, False, "gelu", "f32", 16),
         (300, 512, 1024, 512, True, "gelu_tanh", "f32", 128), (700, 256, 1152, 272, False, "relu", "bf16", 16)]


@pytest.mark.parametrize("M,K,F,N,gated,act,dtype,had", CASES)
def test_against_the_formulas(M, K, F, N, gated, act, dtype, had):
    """Each step from the codes that the step before it left, in 64 bits."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("mlp", M, K, F, N, gated, act, dtype, had)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    block, x, res, dy = _block(torch, M, K, F, N, gated, act, dt, had)
    y = block.forward(x, residual=res)
    c = block.saved
    fc1, fc2 = block.fc1, block.fc2
    qx, sx = qlin.qlin_quantize_rows(x, had_block=had)
    assert torch.equal(qx, c["qx"]) and torch.equal(sx, c["sx"])
    z = qlin.qlin_fwd(qx, sx, fc1.qw, fc1.sw, bias=fc1.bias).cpu()
    codes, scales = ref.checkpoint(z, F)
    assert torch.equal(c["ck"].cpu(), codes) and torch.equal(c["ck_s"].cpu(), scales)
    out = qlin.qlin_fwd(c["qh"], c["sh"], fc2.qw, fc2.sw, bias=fc2.bias)
    assert y.dtype == dt and torch.equal(y, (out + res.float()).to(dt))
    assert torch.equal(block.forward(x, residual=res, save=False), y) and block.saved is c

    dx = block.backward(dy)
    q1, s1, q2, s2, db2 = qlin.qlin_quantize_grad(dy, fc2.sw, c["sh"], want_sum=True)
    assert torch.equal(db2, fc2.db)
    assert torch.equal(fc2.dw, qlin.qlin_bwd_dw(q2, s2, c["qh"]))
    dh = qlin.qlin_bwd_dx(q1, s1, fc2.qw, had_block=had)
    dz, s1, s2, db1 = qlin.qlin_act_bwd(dh, c["ck"], c["ck_s"], act, gated=gated, sw=fc1.sw, sx=sx, dtype=dt,
                                        want_db=True)
    want, err = ref.backward(dh.cpu(), ref.restored(codes, scales, F), F, act)
    off = (dz.double().cpu() - want).abs()
    assert (off <= err + (want.abs() + err) * (ref.STEP[dt] + ref.U)).all()
    assert torch.equal(db1, fc1.db)
    q1, q2 = qlin.qlin_quantize_grad_scaled(dz, fc1.sw, sx, s1, s2)
    assert torch.equal(dx, qlin.qlin_bwd_dx(q1, s1, fc1.qw, had_block=had))
    assert torch.equal(fc1.dw, qlin.qlin_bwd_dw(q2, s2, qx))


def test_gradients_against_differences():
    """The block's input gradient against central differences of its float form (both
    weights as they stand, nothing quantized): they differ by the INT8 rounding of x,
    h and both gradients, each at most half a step of its row's maximum / 127, which
    for normal rows of these lengths is about 1% of the rows' norm; 6% in all is five
    of those in one direction."""
    torch = torch_cuda()
    announce("mlp against differences")
    for gated, act in ((True, "silu"), (False, "gelu")):
        block, x, _, dy = _block(torch, 24, 128, 256, 128, gated, act, torch.float32, seed=3)
        block.forward(x)
        dx = block.backward(dy).double().cpu()
        w1, w2 = (f.unquantized_weight().double().cpu() for f in (block.fc1, block.fc2))
        b1 = block.fc1.bias.double().cpu()

        def loss(v):        # per row
            z = v @ w1.T + b1
            h = ref.act(z[:, :256], act)[0]
            return (((h * z[:, 256:] if gated else h) @ w2.T) * dy.double().cpu()).sum(1)

        v, g = x.double().cpu(), torch.Generator().manual_seed(1)
        for _ in range(8):
            d = torch.randn(v.shape, generator=g, dtype=torch.float64)
            diff = (loss(v + 1e-5 * d) - loss(v - 1e-5 * d)) / 2e-5
            off = ((dx * d).sum(1) - diff).norm() / (dx.norm())
            assert off < 0.06, off      # (a unit-variance direction: the gradient's norm per row)


def test_passes_kept_apart_and_updates():
    torch = torch_cuda()
    announce("mlp: passes kept apart, updates")
    block, x, res, dy = _block(torch, 130, 256, 512, 256, True, "silu", torch.bfloat16)
    other = torch.flip(x, (0,)).contiguous()
    block.forward(x, residual=res)
    first = block.saved
    dx = block.backward(dy)
    dw = block.fc1.dw.clone()
    block.forward(other)
    assert not torch.equal(block.backward(dy), dx)
    assert torch.equal(block.backward(dy, saved=first), dx) and torch.equal(block.fc1.dw, dw)
    before = block.fc1.qw.clone(), block.fc2.qw.clone(), block.fc1.bias.clone()
    block.sgd_step(0.1, 3, 1)
    assert not torch.equal(block.fc1.qw, before[0]) and not torch.equal(block.fc2.qw, before[1])
    assert not torch.equal(block.fc1.bias, before[2])
    block.adamw_step(1e-3, 3, 1)
    block.forward(x[:1].contiguous())
    assert block.backward(dy[:1].contiguous()).shape == (1, 256)


def test_no_tokens():
    torch = torch_cuda()
    announce("mlp: no tokens")
    block, x, res, dy = _block(torch, 5, 128, 256, 128, True, "silu", torch.bfloat16)
    block.forward(x), block.backward(dy)
    y = block.forward(x[:0], residual=res[:0])
    dx = block.backward(dy[:0])
    assert y.shape == (0, 128) and y.dtype == torch.bfloat16 and dx.shape == (0, 128)
    for fc in (block.fc1, block.fc2):
        assert (fc.dw == 0).all() and (fc.db == 0).all()


def test_without_biases():
    """The same as with biases of zeros."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("mlp: no biases")
    g = torch.Generator().manual_seed(8)
    w1, w2, x, dy = (torch.randn(s, generator=g).cuda() for s in ((512, 128), (128, 256), (70, 128), (70, 128)))
    kw = dict(act="gelu", gated=True, dtype=torch.float32)
    plain = qlin.MLPW8A8Training(w1, w2, **kw)
    zeros = qlin.MLPW8A8Training(w1, w2, torch.zeros(512, device="cuda"), torch.zeros(128, device="cuda"), **kw)
    assert torch.equal(plain.forward(x), zeros.forward(x))
    assert torch.equal(plain.backward(dy), zeros.backward(dy))
    assert torch.equal(plain.fc1.dw, zeros.fc1.dw) and torch.equal(plain.fc2.dw, zeros.fc2.dw)
    plain.sgd_step(0.1, 3, 1), zeros.sgd_step(0.1, 3, 1)
    assert torch.equal(plain.fc1.qw, zeros.fc1.qw) and torch.equal(plain.fc2.qw, zeros.fc2.qw)


def test_two_streams_at_once():
    """Passes of one block on streams of their own: each has its workspace."""
    torch = torch_cuda()
    announce("mlp: two streams")
    block, x, res, _ = _block(torch, 600, 4096, 4096, 256, True, "silu", torch.bfloat16)
    inputs = [x, torch.flip(x, (0,)).contiguous()]
    want = [block.forward(v, save=False) for v in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(4):
        got = []
        for s, v in zip(streams, inputs):
            with torch.cuda.stream(s):
                got.append(block.forward(v, save=False))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_block_in_a_graph():
    torch = torch_cuda()
    announce("mlp in a graph")
    block, x, res, dy = _block(torch, 260, 256, 2304, 256, True, "gelu_tanh", torch.bfloat16)
    want = block.forward(x, residual=res), block.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.forward(x, residual=res)
        dx = block.backward(dy)
    for _ in range(3):
        y.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        block.forward(torch.zeros_like(x))          # the program's own work in between
        torch.cuda.synchronize()


def test_refusals():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    w1, w2 = torch.randn(64, 32).cuda(), torch.randn(32, 64).cuda()
    with pytest.raises(ValueError):
        qlin.MLPW8A8Training(w1, w2, gated=True, had_block=16)
    with pytest.raises(ValueError):
        qlin.MLPW8A8Training(w1, w2, act="swish", had_block=16)
    block = qlin.MLPW8A8Training(w1, w2, had_block=16)
    with pytest.raises(RuntimeError):
        block.backward(torch.zeros((4, 32), device="cuda"))
