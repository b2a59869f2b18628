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
