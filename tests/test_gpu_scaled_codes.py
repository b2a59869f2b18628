"""qlin_quantize_grad_scaled where a scale is not the maximum of the gradient that it is
given: codes stay within +-127, with the value's sign."""
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def test_a_gradient_that_is_subnormal_in_bf16():
    """dz = 1.6 2^-133 rounds to 2^-132 in bf16, a quarter more than the value that s1
    and s2 are from: with weights and tokens of large scales the quotients are about 159,
    and the codes 127."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("subnormal bf16 gradient")
    M, N = 40, 64
    dy = torch.full((M, N), 1.6 * 2.0 ** -133, dtype=torch.float32)
    dy[:, 1::2] *= -1
    dy[3] = 0.0
    ck, ck_s = torch.ones((M, N), dtype=torch.int8), torch.ones((M, N // 32))
    sw, sx = torch.full((N,), 2.0 ** 40), torch.full((M,), 2.0 ** 44)
    sw, sx = sw.cuda(), sx.cuda()
    dz, s1, s2, _ = qlin.qlin_act_bwd(dy.cuda(), ck.cuda(), ck_s.cuda(), "none", sw=sw, sx=sx)
    assert (dz[0, 0].double() == 2.0 ** -132) and bool((s1[[0, 1, 2]] > 2.0 ** -126).all())
    q1, q2 = qlin.qlin_quantize_grad_scaled(dz, sw, sx, s1, s2)
    want = torch.full((M, N), 127, dtype=torch.int8)
    want[:, 1::2] = -127
    want[3] = 0
    assert torch.equal(q1.cpu(), want) and torch.equal(q2.cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(1, 16), (40, 528)])
def test_scales_that_are_too_small(dtype, M, N):
    """Saturated codes, and every other one as for larger scales' values: round to nearest,
    ties to even, of the quotient, whose own roundings are 3 2^-24 of it."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("small scales", dtype, M, N)
    g = torch.Generator().manual_seed(3)
    dy = torch.randn((M, N), generator=g).to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    sw, sx = torch.rand(N, generator=g) + 0.5, torch.rand(M, generator=g) + 0.5
    s1, s2 = torch.full((M,), 2.0 ** -7), torch.full((N,), 2.0 ** -7)
    s1[M // 2], s2[5] = 2.0 ** -60, 2.0 ** -40
    q1, q2 = qlin.qlin_quantize_grad_scaled(dy.cuda(), sw.cuda(), sx.cuda(), s1.cuda(), s2.cuda())
    for q, by, s in ((q1, sw[None], s1[:, None]), (q2, sx[:, None], s2[None])):
        v = (dy.double() * by.double() / s.double()).clamp(-127, 127)
        assert ((q.cpu().double() - v).abs() <= 0.5 + 3 * 2.0 ** -24 * 127.5).all()
        assert int((v.abs() == 127).sum()) > 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_that_are_not_finite(dtype):
    """The same codes as qlin_quantize_grad's, for the scales that it gives such a gradient."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N = 64, 272
    g = torch.Generator().manual_seed(5)
    sw, sx = (torch.rand(N, generator=g) + 0.5).cuda(), (torch.rand(M, generator=g) + 0.5).cuda()
    for bad in (float("nan"), float("inf"), -float("inf")):
        announce("codes of", bad, dtype)
        dy = torch.randn((M, N), generator=g).to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
        dy[3, 7] = dy[40, 100] = dy[41, 100] = bad
        dy = dy.cuda()
        q1, s1, q2, s2, _ = qlin.qlin_quantize_grad(dy, sw, sx)
        c1, c2 = qlin.qlin_quantize_grad_scaled(dy, sw, sx, s1, s2)
        assert torch.equal(c1, q1) and torch.equal(c2, q2)
