"""The products with an activation where a width ends inside a checkpoint's block."""
import pytest

from tests import block_ref as ref
from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 8, 40, 700])
@pytest.mark.parametrize("gated", [False, True])
def test_the_last_block_is_its_own_outputs(M, gated):
    """The gate's last block has 16 outputs; the rows of the weight behind its own are
    the other half's, whose sums times the row's scale are past fp32 here."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("last block", M, gated)
    F, K = 48, 256
    N = 2 * F if gated else F
    qx = torch.full((M, K), 127, dtype=torch.int8)
    qw = torch.zeros((N, K), dtype=torch.int8)
    qw[torch.arange(F), torch.arange(F)] = torch.arange(-24, 24, dtype=torch.int8)
    qw[F:] = 127
    sx, sw = torch.full((M,), 1e33), torch.full((N,), 1e-34)
    args = [t.cuda() for t in (qx, sx, qw, sw)]
    z = qlin.qlin_fwd(*args).cpu()
    assert z[:, :F].isfinite().all() and not z[:, F:].isfinite().any()
    first = qlin.qlin_fwd_gated if gated else qlin.qlin_fwd_act
    _, ck, ck_s = first(*args, act="silu", save=True)
    codes, scales = ref.checkpoint(z[:, :F].contiguous(), F)
    assert torch.equal(ck_s[:, :2].cpu(), scales) and torch.equal(ck[:, :F].cpu(), codes)
    assert not ck_s[:, 2:].isfinite().any()
