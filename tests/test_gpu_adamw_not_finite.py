"""Infinite gradients, and an epsilon below the smallest normal number."""
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu
STEP = (1e-3, 0.9, 0.999, 1e-8, 1)      # learning rate, betas, epsilon, seed


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_8_bit_block_with_an_infinity_or_nan(value):
    """Both scales of the block become NaN at once, whichever it was, and the blocks
    beside it go on as if nothing were there."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("8-bit block", value)
    g = torch.Generator().manual_seed(2)
    n = 256 * 5 + 17

    def fresh():
        g.manual_seed(2)
        r = lambda *s: torch.randn(s, generator=g).cuda()               # noqa: E731
        return dict(p=r(n), g=r(n), m=r(n).to(torch.float8_e4m3fn), v=r(n).abs().to(torch.float8_e4m3fn),
                    m_scale=r(6).abs() * 1e-3, v_scale=r(6).abs() * 1e-3)

    t, ref = fresh(), fresh()
    t["g"][2 * 256 + 9] = value
    ours, plain = qlin.qlin_adamw_tensors_plan([t]), qlin.qlin_adamw_tensors_plan([ref])
    other = torch.ones(n, dtype=torch.bool, device="cuda")
    other[512:768] = False
    for step in (1, 2):
        for plan in (ours, plain):
            qlin.qlin_adamw_tensors(plan, *STEP, step)
        assert t["m_scale"].isnan().nonzero().tolist() == [[2]]
        assert t["v_scale"].isnan().nonzero().tolist() == [[2]]
        for k in ("p", "m", "v"):
            assert torch.equal(t[k].float()[other], ref[k].float()[other])
        for k in ("m_scale", "v_scale"):
            assert torch.equal(t[k][[0, 1, 3, 4, 5]], ref[k][[0, 1, 3, 4, 5]])
        t["g"][2 * 256 + 9] = 0.0
    assert t["p"][512:768].isnan().all()


@pytest.mark.parametrize("eps", [1e-38, 1e-39, 1e-44])
@pytest.mark.parametrize("bits", [32, 8])
def test_epsilon_below_the_normal_numbers(eps, bits):
    """Elements that have never had a gradient stay where they are (0 / eps), others
    move by m' / (root + eps), where eps is nothing."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("epsilon", eps, bits)
    n = 700
    zeros = lambda k, t=torch.float32: torch.zeros(k, device="cuda").to(t)     # noqa: E731
    kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
    t = dict(p=torch.ones(n, device="cuda"), g=zeros(n), m=zeros(n, kind), v=zeros(n, kind))
    if bits == 8:
        t["m_scale"], t["v_scale"] = zeros(3), zeros(3)
    t["g"][::2] = 0.25
    qlin.qlin_adamw_tensors(qlin.qlin_adamw_tensors_plan([t]), 1e-3, 0.9, 0.999, eps, 1, 1)
    assert (t["p"][1::2] == 1).all()
    # the first step is lr whatever the gradient, within the roundings of m', v', their
    # root and quotient and of the constants: 32 of 2^-24 of the step, one of p
    assert ((t["p"][::2].double() - (1 - 1e-3)).abs() <= 32 * 2.0 ** -24 * 1e-3 + 2.0 ** -24).all()
