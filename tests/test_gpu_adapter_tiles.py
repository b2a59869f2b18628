"""The products that add the adapters' term in their own epilogues: outputs of 128
tiles of 256 x 256 or more, with ragged edges, ranks that do not fill a step, tiles
whose tokens have one, several or no adapters, and a split last round of tiles.
The references, bounds and their derivation are those of the smaller shapes."""
import pytest

from tests import test_gpu_adapter as small
from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu

FWD = [(2100, 4112, 96, 3, 32), (2081, 4112, 80, 40, 8), (2100, 4112, 96, 5, 24),
       (4500, 2064, 64, 2, 128), (2100, 8208, 1536, 3, 16)]
BWD = [(2100, 96, 4096, 3, 16, 128), (1100, 48, 8192, 2, 128, 64), (2081, 80, 4112, 40, 8, 16),
       (4500, 64, 2064, 5, 40, 0), (2100, 64, 4096, 3, 32, 512), (2100, 1536, 8208, 3, 16, 16)]


@pytest.mark.parametrize("M,N,K,L,R", FWD)
@pytest.mark.parametrize("w", ["f32", "bf16"])
@pytest.mark.parametrize("runs", [None, 4])
def test_forward(M, N, K, L, R, w, runs):
    small.test_forward(M, N, K, L, R, w, runs)


@pytest.mark.parametrize("M,N,K,L,R,had", BWD)
@pytest.mark.parametrize("w,dy", [("f32", "f32"), ("bf16", "bf16")])
def test_backward(M, N, K, L, R, had, w, dy):
    small.test_backward(M, N, K, L, R, had, w, dy)


@pytest.mark.parametrize("dy", ["f32", "bf16"])
def test_backward_of_many_ranks(dy):
    """Enough tokens and ranks that 32 ranks share the read of dY."""
    small.test_backward(4112, 64, 2064, 2, 128, 16, "bf16", dy)


@pytest.mark.parametrize("w", ["f32", "bf16"])
def test_backward_of_mixed_tokens(w):
    """Every 16-token block of the product holds several adapters."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K, L, R = 2100, 64, 4112, 4, 24
    announce("mixed", w)
    c = small._case(torch, M, N, K, L, R, w, "f32", seed=6)
    c["u"] = torch.randn((M, R), generator=torch.Generator().manual_seed(1))
    d = small._cuda(c)
    dx, da, db = small._run_bwd(qlin, d, L)
    dx64 = (c["qg"].double() @ c["qw"].double()) * c["sg"].double()[:, None]
    base, low = dx64.abs(), torch.zeros_like(dx64)
    for l in range(L):
        at = torch.nonzero(c["ids"] == l)[:, 0]
        A, B, sc = c["a"][l].double(), c["b"][l].double(), c["scale"][l].double()
        D = c["dy"][at].double()
        dx64[at] += (sc * (D @ B)) @ A
        low[at] += (sc * (D.abs() @ B.abs())) @ A.abs()
    bound = 16 * small.U * (base + low) + low * (2 * small.SPLIT + (N + R + 64) * small.U)
    assert ((dx.double().cpu() - dx64).abs() <= bound).all()


@pytest.mark.parametrize("w", ["f32", "bf16"])
def test_values_of_other_adapters_do_not_reach_a_token(w):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("isolation", w)
    M, N, K, L, R = 2100, 4112, 4112, 3, 16
    c = small._case(torch, M, N, K, L, R, w, "f32", seed=5)
    d = small._cuda(c)
    y, d["u"] = small._run_fwd(qlin, d)
    dx, _, _ = small._run_bwd(qlin, d, L, 16)
    d["a"][1, 3, 5] = float("nan")
    d["b"][1, 7, 1] = float("inf")
    y2, _ = small._run_fwd(qlin, d)
    dx2, _, _ = small._run_bwd(qlin, d, L, 16)
    other = d["ids"] != 1
    assert torch.equal(y[other], y2[other]) and torch.equal(dx[other], dx2[other])
    assert y2[~other].isnan().any(1).all() and dx2[~other].isnan().any(1).all()
