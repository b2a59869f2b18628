"""The layer that runs the norm, the adapters and the optimizer together, and the
example that trains it."""
import os
import sys

import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _layer(torch, had=64, dtype=None, bits=32, K=256, N=192):
    from w8a8_integer_linear_amd import AdaptedLinearW8A8
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g).cuda()               # noqa: E731
    adapters = [(r(5, K) * 0.1, r(N, 5) * 0.1, 10.0), (r(16, K) * 0.1, r(N, 16) * 0.1, 16.0)]
    return AdaptedLinearW8A8(r(N, K) * 0.05, 1 + 0.1 * r(K), adapters, bias=r(N), had_block=had,
                             dtype=dtype or torch.float32, state_bits=bits), adapters


@pytest.mark.parametrize("had", [0, 64])
def test_adapters_come_back_in_the_original_basis(had):
    torch = torch_cuda()
    layer, adapters = _layer(torch, had)
    assert layer.R == 16 and (layer.a[0, 5:] == 0).all() and (layer.b[0, :, 5:] == 0).all()
    assert torch.equal(layer.scale.cpu(), torch.tensor([2.0, 1.0]))
    for l, (A, B, _) in enumerate(adapters):
        A2, B2 = layer.adapter(l)
        # two rotations of 64 in fp32: 14 roundings of sums of 8 times the size
        assert (A2 - A).abs().max() <= 14 * 8 * 2.0 ** -24 * A.abs().max() * 8
        assert torch.equal(B2, B)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_forward_and_gradients(M):
    """The step's values against autograd in 64 bits over the values that the
    layer's own codes stand for."""
    torch = torch_cuda()
    announce("adapted layer", M)
    layer, _ = _layer(torch)
    g = torch.Generator().manual_seed(M)
    x, res = (torch.randn((M, 256), generator=g).cuda() for _ in range(2))
    ids = torch.randint(-1, 2, (M,), generator=g, dtype=torch.int32).cuda()
    dres, dy = torch.randn((M, 256), generator=g).cuda(), torch.randn((M, 192), generator=g).cuda()
    y, h = layer.forward(x, ids, residual=res)
    y, h = y.clone(), h.clone()
    c = layer._buffers[(M, torch.float32)]
    dh = layer.backward(dy, dres=dres)
    D = torch.float64
    had = layer.had
    H = torch.ones((1, 1), dtype=D)
    while H.shape[0] < had:
        H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)])
    H = (H / had ** 0.5).cuda()
    rot = lambda t: (t.reshape(-1, had) @ H).reshape(t.shape)           # noqa: E731
    xq = c["qx"].to(D) * c["sx"].to(D)[:, None]
    W = layer.qw.to(D) * layer.sw.to(D)[:, None]
    a, b = layer.a.to(D).requires_grad_(), layer.b.to(D).requires_grad_()
    ok = (ids >= 0)
    A, B = a[ids.clamp(0).long()], b[ids.clamp(0).long()]
    sc = (layer.scale[ids.clamp(0).long()] * ok).to(D)
    xr = xq.clone().requires_grad_()
    u = (A * xr[:, None, :]).sum(2) * sc[:, None]
    want = xr @ W.T + layer.bias.to(D) + (B * u[:, None, :]).sum(2)
    assert (y.to(D) - want).abs().max() <= 2.0 ** -18 * want.abs().max()
    want.backward(dy.to(D))
    for got, ref in ((layer.da, a.grad), (layer.db, b.grad)):
        assert (got.to(D) - ref).norm() <= 2.0 ** -16 * max(ref.norm().item(), 1e-6)
    # dx: the frozen weight's part takes dY's INT8 codes, half a step off each
    gq = (c["qg"].to(D) * c["sg"].to(D)[:, None])
    dn = rot(gq @ layer.qw.to(D) + xr.grad - dy.to(D) @ W)
    h64 = h.to(D).requires_grad_()
    gamma = layer.gamma.to(D).requires_grad_()
    n = h64 * torch.rsqrt(h64.square().mean(1, keepdim=True) + layer.eps) * gamma
    n.backward(dn)
    ref = h64.grad + dres.to(D)
    assert (dh.to(D) - ref).norm() <= 2.0 ** -16 * ref.norm()
    assert (layer.dgamma.to(D) - gamma.grad).norm() <= 2.0 ** -16 * gamma.grad.norm()


def test_steps_of_several_sizes_share_the_layer():
    """Prompts, single tokens and training batches in turn give what a fresh layer
    gives for each."""
    torch = torch_cuda()
    layer, _ = _layer(torch)
    g = torch.Generator().manual_seed(3)
    for M in (300, 1, 17, 300, 600, 1):
        x = torch.randn((M, 256), generator=g).cuda()
        ids = torch.randint(-1, 2, (M,), generator=g, dtype=torch.int32).cuda()
        dy = torch.randn((M, 192), generator=g).cuda()
        y = layer.forward(x, ids)[0].clone()
        dh = layer.backward(dy).clone()
        other, _ = _layer(torch)
        assert torch.equal(y, other.forward(x, ids)[0])
        assert torch.equal(dh, other.backward(dy))
        assert torch.equal(layer.da, other.da) and torch.equal(layer.db, other.db)


def test_refusals():
    torch = torch_cuda()
    from w8a8_integer_linear_amd import pack_adapters
    A, B = torch.zeros((4, 64), device="cuda"), torch.zeros((32, 4), device="cuda")
    for bad in ([], [(A, torch.zeros((32, 5), device="cuda"), 1.0)],
                [(torch.zeros((129, 64), device="cuda"), torch.zeros((32, 129), device="cuda"), 1.0)],
                [(A, B, 1.0), (torch.zeros((4, 48), device="cuda"), B, 1.0)]):
        with pytest.raises(ValueError):
            pack_adapters(bad)
    layer, _ = _layer(torch)
    with pytest.raises(TypeError):
        layer.forward(torch.zeros((3, 256), device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("bits,bf16", [(32, False), (8, False), (32, True), (8, True)])
def test_example_trains_every_adapter(bits, bf16):
    torch_cuda()
    announce("finetune_adapters", bits, bf16)
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import finetune_adapters
    finally:
        sys.path.pop(0)
    losses, layer, error = finetune_adapters.train(steps=120, state_bits=bits, bf16=bf16,
                                                  say=lambda *a: None)
    assert losses[-1] < 0.05 * losses[0]
    assert max(error) < 0.15
