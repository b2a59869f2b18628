"""What the adapted layer keeps between its calls, and whose its results are."""
import pytest

from tests.gpu_util import announce, torch_cuda
from tests.test_gpu_adapted_layer import _layer

pytestmark = pytest.mark.gpu


def _batch(torch, M, seed, dtype=None):
    g = torch.Generator().manual_seed(seed)
    x, res = (torch.randn((M, 256), generator=g).to(dtype or torch.float32).cuda() for _ in range(2))
    ids = torch.randint(-1, 2, (M,), generator=g, dtype=torch.int32).cuda()
    return x, ids, res, torch.randn((M, 192), generator=g).cuda()


def _alone(torch, batch):
    """A fresh layer's results for one batch."""
    x, ids, res, dy = batch
    layer, _ = _layer(torch)
    y, h = layer.forward(x, ids, residual=res)
    return y, h, layer.backward(dy), layer.da, layer.db, layer.dgamma


def test_memory_stays_bounded_over_token_counts():
    torch = torch_cuda()
    layer, _ = _layer(torch)
    batches = [_batch(torch, M, M) for M in range(1, 121)]

    def step(x, ids, res, dy):
        announce("layer of", x.shape[0])
        layer.forward(x, ids, residual=res)
        layer.backward(dy)

    step(*batches[-1])
    before = torch.cuda.memory_allocated()
    for b in batches:
        step(*b)
    assert torch.cuda.memory_allocated() <= before + (1 << 16)


def test_results_belong_to_the_caller():
    torch = torch_cuda()
    layer, _ = _layer(torch)
    a, b = _batch(torch, 40, 1), _batch(torch, 40, 2)
    kept, want = [], []
    for x, ids, res, dy in (a, b):
        y, h = layer.forward(x, ids, residual=res)
        kept += [y, h, layer.backward(dy)]
        want += [t.clone() for t in kept[-3:]]
    for t, w in zip(kept, want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("MA,MB", [(40, 40), (300, 17)])
def test_backward_of_an_earlier_forward(MA, MB):
    """Two forward passes, then both backward passes, the first one's last."""
    torch = torch_cuda()
    layer, _ = _layer(torch)
    a, b = _batch(torch, MA, 1), _batch(torch, MB, 2)
    saved = []
    for x, ids, res, _ in (a, b):
        layer.forward(x, ids, residual=res)
        saved.append(layer.saved)
    for batch, c in ((b, None), (a, saved[0]), (b, saved[1])):
        dh = layer.backward(batch[3], saved=c)
        _, _, dh1, da, db, dgamma = _alone(torch, batch)
        for t, w in zip((dh, layer.da, layer.db, layer.dgamma), (dh1, da, db, dgamma)):
            assert torch.equal(t, w)


def test_serving_between_forward_and_backward():
    torch = torch_cuda()
    layer, _ = _layer(torch)
    a, b = _batch(torch, 40, 1), _batch(torch, 40, 2)
    layer.forward(a[0], a[1], residual=a[2])
    y, h = layer.forward(b[0], b[1], residual=b[2], save=False)
    want = _alone(torch, b)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    dh, want = layer.backward(a[3]), _alone(torch, a)
    for t, w in zip((dh, layer.da, layer.db, layer.dgamma), want[2:]):
        assert torch.equal(t, w)


def test_backward_needs_a_forward():
    torch = torch_cuda()
    layer, _ = _layer(torch)
    x, ids, res, dy = _batch(torch, 5, 1)
    layer.forward(x, ids, residual=res, save=False)
    with pytest.raises(RuntimeError):
        layer.backward(dy)


def _long(torch, M, seed):
    """A layer whose products split their contraction (their workgroups meet in the
    workspace), and a batch for it."""
    layer, _ = _layer(torch, K=2048, N=512)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, 2048), generator=g).cuda()
    ids = torch.randint(-1, 2, (M,), generator=g, dtype=torch.int32).cuda()
    return layer, x, ids, torch.randn((M, 512), generator=g).cuda()


def test_streams_do_not_share_a_workspace():
    torch = torch_cuda()
    announce("two streams")
    layer, xa, ids, _ = _long(torch, 400, 1)
    xb = xa.flip(0).contiguous()
    want = [layer.forward(x, ids)[0] for x in (xa, xb)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = ([], [])
    for _ in range(20):
        for k, x in enumerate((xa, xb)):
            with torch.cuda.stream(side[k]):
                got[k].append(layer.forward(x, ids, save=False)[0])
    torch.cuda.synchronize()
    for k in range(2):
        for y in got[k]:
            assert torch.equal(y, want[k])


def test_graphs_keep_their_workspace():
    """Graphs captured before and after eager calls, which grow the layer's workspace
    between the replays."""
    torch = torch_cuda()
    announce("graphs of the layer")
    layer, x, ids, dy = _long(torch, 400, 2)
    graphs = []

    def capture():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, _ = layer.forward(x, ids)
            dh = layer.backward(dy)
        graphs.append((graph, y, dh))

    capture()
    for k, M in enumerate((100, 900, 2000)):
        _, big, many, grad = _long(torch, M, 3)
        x.copy_(torch.randn(x.shape, device="cuda"))
        layer.forward(big, many)
        layer.backward(grad)
        want = [layer.forward(x, ids)[0], layer.backward(dy), layer.da.clone(), layer.db.clone()]
        torch.cuda.synchronize()
        for graph, y, dh in graphs:
            for t in (y, dh, layer.da, layer.db):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip((y, dh, layer.da, layer.db), want):
                assert torch.equal(a, b)
        capture()


@pytest.mark.parametrize("bits", [32, 8])
def test_weight_decay_may_change(bits):
    """Without gradients a step is the decay alone: p (1 - lr wd), two roundings.  With
    them, the moments go on as without any decay."""
    torch = torch_cuda()
    announce("weight decay", bits)
    layer, plain = (_layer(torch, bits=bits)[0] for _ in range(2))
    lr, step = 1e-2, 0
    for decay in (0.0, 0.5, 0.5, 0.25, 0.0):
        step += 1
        before = [t.clone() for t in (layer.a, layer.b, layer.gamma)]
        layer.adamw_step(lr, seed=3, step=step, weight_decay=decay)
        plain.adamw_step(lr, seed=3, step=step)
        for p, old, wd in zip((layer.a, layer.b, layer.gamma), before, (decay, decay, 0.0)):
            want = old.double() * (1 - lr * wd)
            assert ((p.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all()
    g = torch.Generator(device="cuda").manual_seed(1)
    for decay in (0.1, 0.0, 0.2):
        step += 1
        for a, b in zip((layer.da, layer.db, layer.dgamma), (plain.da, plain.db, plain.dgamma)):
            a.normal_(generator=g)
            b.copy_(a)
        layer.adamw_step(lr, seed=3, step=step, weight_decay=decay)
        plain.adamw_step(lr, seed=3, step=step)
    for t, u in zip(layer._trained, plain._trained):
        for k in set(t) - {"p", "g", "weight_decay"}:
            assert torch.equal(t[k].float(), u[k].float()) and (t[k].float() != 0).any()
