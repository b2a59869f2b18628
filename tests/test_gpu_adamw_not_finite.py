"""Infinite gradients and NaN in the moments held in 8 bits."""
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
