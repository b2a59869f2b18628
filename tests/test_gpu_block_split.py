"""Products with an activation whose last round of tiles is split along the contraction:
every activation, residuals, and the workspaces that the binding itself makes, whose
arrival counters it clears: eager, on two streams at once and in captured graphs."""
import pytest

from tests import block_ref as ref
from tests.gpu_util import announce, torch_cuda
from tests.test_gpu_block import ACTS, _near, _operands

pytestmark = pytest.mark.gpu

# All tiles in two pieces; in three; whole rounds before the split one.
SHAPES = [(600, 8160, 4112), (900, 2112, 2064), (1300, 11744, 1552)]


def _sizes(qlin, M, N, K):
    need = [qlin.qlin_fwd_act_ws_bytes(M, N, K), qlin.qlin_fwd_gated_ws_bytes(M, N // 2, K)]
    assert all(n > 4096 for n in need)
    return need


def _dirty(torch, *sizes):
    """Blocks of these sizes, full of ones, that the allocator hands out next."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    at = {t.data_ptr() for t in held}
    del held
    return at


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_activations_and_residuals(M, N, K, act):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    need, F = _sizes(qlin, M, N, K), N // 2
    qx, sx, qw, sw, b = _operands(torch, M, N, K, 7)
    z = qlin.qlin_fwd(qx, sx, qw, sw, bias=b).cpu()
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(2)
    for y_type, r_type, place in ((torch.float32, torch.float32, True), (torch.bfloat16, torch.bfloat16, True),
                                  (torch.float32, torch.bfloat16, False), (torch.bfloat16, torch.float32, False)):
        announce("split act", M, N, K, act, y_type, r_type, place)
        res = (3 * torch.randn((M, N), generator=g)).to(r_type)
        want, err = ref.forward(z, N, act, res)
        r = res.cuda()
        y, ck, ck_s = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, act=act, residual=r, y=r if place else None,
                                        dtype=y_type, save=True, workspace=ws)
        assert not place or y is r
        _near(torch, y, want, err, (y_type, r_type))
        codes, scales = ref.checkpoint(z, N)
        assert torch.equal(ck.cpu(), codes) and torch.equal(ck_s.cpu(), scales)
        announce("split gated", M, F, K, act, y_type)
        want, err = ref.forward(z, F, act)
        y = qlin.qlin_fwd_gated(qx, sx, qw, sw, bias=b, act=act, dtype=y_type, workspace=ws)[0]
        _near(torch, y, want, err, y_type)
    assert bool((ws[:4096] == 0).all())         # the counters, for the next call


def _calls(qlin, ops, stream=None):
    qx, sx, qw, sw, b = ops
    a = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, act="gelu", save=True, stream=stream)
    g = qlin.qlin_fwd_gated(qx, sx, qw, sw, bias=b, act="silu", save=True, stream=stream)
    return *a, *g


def _wanted(torch, qlin, ops):
    """The same with the caller's workspace, zero-filled."""
    qx, sx, qw, sw, b = ops
    ws = torch.zeros(max(_sizes(qlin, *qx.shape[:1], *qw.shape)), dtype=torch.uint8, device="cuda")
    a = qlin.qlin_fwd_act(qx, sx, qw, sw, bias=b, act="gelu", save=True, workspace=ws)
    g = qlin.qlin_fwd_gated(qx, sx, qw, sw, bias=b, act="silu", save=True, workspace=ws)
    return *a, *g


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_the_bindings_own_workspace(M, N, K, monkeypatch):
    """Made from memory that held something else: its counters are cleared."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    from w8a8_integer_linear_amd import _native as nat
    ops = _operands(torch, M, N, K, 3)
    want = _wanted(torch, qlin, ops)
    made = []
    scratch = nat._scratch
    monkeypatch.setattr(nat, "_scratch", lambda *a: made.append(scratch(*a)) or made[-1])
    for _ in range(3):
        announce("own workspace", M, N, K)
        made.clear()
        old = _dirty(torch, *_sizes(qlin, M, N, K))
        got = _calls(qlin, ops)
        torch.cuda.synchronize()
        assert len(made) == 2 and made[0].data_ptr() in old         # (the memory just filled)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(bool((m[:4096] == 0).all()) for m in made)


def test_two_streams_at_once():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K = SHAPES[0]
    announce("split tiles on two streams at once")
    sets = [_operands(torch, M, N, K, k) for k in (1, 2)]
    want = [_wanted(torch, qlin, o) for o in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    _dirty(torch, *_sizes(qlin, M, N, K))
    for _ in range(4):
        got = [_calls(qlin, o, stream=s) for o, s in zip(sets, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_replayed_graph(M, N, K):
    """Its workspaces are made, and cleared, in the capture; every replay clears them."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    ops = _operands(torch, M, N, K, 2)
    sets = [_operands(torch, M, N, K, s) for s in (2, 12, 22)]
    want = [_wanted(torch, qlin, o) for o in sets]
    torch.cuda.synchronize()
    announce("split tiles in a graph", M, N, K)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _calls(qlin, ops)
    for k in (0, 1, 2, 0):
        for t, v in zip(ops, sets[k]):
            t.copy_(v)
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[k], held)), k
        _calls(qlin, sets[k])           # the program's own work in between
        torch.cuda.synchronize()


def test_layer_in_a_graph():
    """Forward and backward of a layer whose products split their tiles."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, K, F, N = 600, 4112, 4080, 256
    g = torch.Generator().manual_seed(4)
    r = lambda *s, std=1.0: (std * torch.randn(s, generator=g)).cuda()        # noqa: E731
    block = qlin.MLPW8A8Training(r(2 * F, K, std=K ** -0.5), r(N, F, std=F ** -0.5), r(2 * F), r(N), act="gelu",
                                 gated=True, had_block=16)
    _sizes(qlin, M, 2 * F, K)
    x, dy = r(M, K).bfloat16(), r(M, N, std=0.1)
    want = block.forward(x), block.backward(dy)
    torch.cuda.synchronize()
    announce("layer with split tiles in a graph")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.forward(x)
        dx = block.backward(dy)
    for _ in range(3):
        y.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        block.forward(torch.zeros_like(x), save=False)
        torch.cuda.synchronize()
