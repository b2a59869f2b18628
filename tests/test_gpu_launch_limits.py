"""Row and chunk counts whose threads no single launch can hold (2^32 per grid
dimension): the calls around the projection answer them like any other."""
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def test_norm_of_2_24_rows():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    rows, cols = (1 << 24) + 3, 16
    announce("rmsnorm_quant", rows, cols)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16)
    gamma = torch.rand(cols, generator=g, device="cuda") + 0.5
    got = qlin.qlin_rmsnorm_quant(x, gamma, 1e-6, residual=res, had_block=16, want_y=True)
    step = 5_000_000        # (pieces that do not end where a launch may)
    for at in range(0, rows, step):
        part = slice(at, min(rows, at + step))
        want = qlin.qlin_rmsnorm_quant(x[part], gamma, 1e-6, residual=res[part], had_block=16,
                                       want_y=True)
        for a, b in zip(got, want):
            assert torch.equal(a[part], b)
