"""The activations' values and derivatives at chosen z, through the products' epilogues
and the backward pass: z is the bias where the row's scale is 0, and a checkpoint's
scale times 1.

Bounds relative to the value, from the kernels' arithmetic (U = 2^-24, the hardware's
exp2 and reciprocal within 2 U):
  gelu  Phi(-x), x = |z|, is t P(t) e^(-x^2 / 2), t = 1 / (1 + 0.34 x): the fit 0.7 U,
        eight Horner steps (partial sums over the sum, at most 3.1) 3.1 U, t's 3 U through
        a slope of at most 2.4, 7.1 U, exp2 2 U, two products 2 U: less than 16 U together.
        The exponent's two roundings and its constant's, 3 U of x^2 / 2.  z Phi(z) for z < 0
        is one more product; for z > 0 it is z - z Phi(-z).
  An exponential below 2^-126 may be flushed, at x >= 13.2: 2^-120 in all."""
import math

import pytest

from tests import block_ref as ref
from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu
U = ref.U
TINY = ref.TINY


def _points(torch):
    """8192 fp32 values: an even grid over +-14, both tails, around 0, and far out."""
    g = torch.linspace(-14.0, 14.0, 4096)
    tails = torch.cat([torch.linspace(-8.0, -2.0, 2048), torch.linspace(-2.0, 0.0, 1024)])
    tiny = torch.cat([s * 2.0 ** -torch.arange(1.0, 101.0) for s in (-1.0, 1.0)])
    far = torch.cat([s * 2.0 ** torch.arange(4.0, 104.0) for s in (-1.0, 1.0)])
    z = torch.cat([g, tails, tiny, far, torch.zeros(1)])
    return torch.cat([z, torch.linspace(-1.0, 1.0, 8192 - len(z))])


def _gelu(torch, z):
    """(z Phi(z), its error) in 64 bits."""
    z, x = z.double(), z.double().abs()
    q = torch.special.erfc(x * math.sqrt(0.5)) / 2
    eq = q * (16 * U + x * x * 1.5 * U) + TINY
    v = torch.where(z > 0, z - z * q, z * q)
    return v, x * eq + 2 * U * v.abs() + TINY


@pytest.mark.parametrize("path,M,save", [("streamed", 3, False), ("few tokens", 3, True),
                                         ("few tokens", 40, False), ("tiles", 700, False)])
def test_gelu_values(path, M, save):
    """Everywhere to a few units of the value's own last place, its tail included: below
    -6 it falls on to 0."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    z = _points(torch)
    N, K = len(z), 64
    announce("gelu", path, M, save)
    zeros = torch.zeros((M, K), dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    y = qlin.qlin_fwd_act(*zeros, *w, bias=z.cuda(), act="gelu", dtype=torch.float32, save=save)[0]
    want, err = _gelu(torch, z)
    off = (y.double().cpu() - want).abs()
    assert (off <= err).all(), (z[(off > err).any(0)][:8], float((off / err).max()))


def test_gelu_values_of_the_backward_pass():
    """The other half's gradient is dy act(z), the same function as the forward's."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    z = _points(torch)
    M, F = len(z), 32           # a row and its one block per z
    announce("gelu, backward")
    ck = torch.ones((M, 2 * F), dtype=torch.int8)
    ck[z < 0] = -1
    ck_s = z.abs()[:, None].expand(M, 2).contiguous()
    dy = torch.ones((M, F), device="cuda")
    dz = qlin.qlin_act_bwd(dy, ck.cuda(), ck_s.cuda(), "gelu", gated=True, dtype=torch.float32)[0]
    want, err = _gelu(torch, z)
    off = (dz[:, F].double().cpu() - want).abs()
    assert (off <= err).all(), float((off / err).max())


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_far_from_zero(act, gated):
    """Where an activation has become z or 0, so has its derivative 1 or 0, up to the
    largest z: also where z^2 is past fp32."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("far from zero", act, gated)
    z = torch.cat([s * 2.0 ** torch.arange(7.0, 127.0) for s in (-1.0, 1.0)])
    M, F = len(z), 32
    N = 2 * F if gated else F
    ck = torch.ones((M, N), dtype=torch.int8)
    ck[:, :F][z < 0] = -1
    ck_s = torch.ones((M, N // 32))
    ck_s[:, 0] = z.abs()
    dz, s1, s2, db = qlin.qlin_act_bwd(torch.ones((M, F), device="cuda"), ck.cuda(), ck_s.cuda(), act, gated=gated,
                                       sw=torch.ones(N, device="cuda"), sx=torch.ones(M, device="cuda"),
                                       dtype=torch.float32, want_db=True)
    on = torch.ones(M, dtype=torch.double) if act == "none" else (z > 0).double()
    dz = dz.double().cpu()
    assert ((dz[:, :F] - on[:, None]).abs() <= TINY).all()
    if gated:
        assert ((dz[:, F:] - (z.double() * on)[:, None]).abs() <= TINY).all()
    assert s1.isfinite().all() and s2.isfinite().all() and db.isfinite().all()


def test_the_largest_checkpoint():
    """z next to fp32's largest: its block's scale times 128 is past fp32."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("largest checkpoint")
    M, N, K = 3, 64, 64
    b = torch.linspace(-1.0, 1.0, N)
    b[:32] = 0.999 * torch.finfo(torch.float32).max
    b[7] *= -1
    zeros = torch.zeros((M, K), dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    y, ck, ck_s = qlin.qlin_fwd_act(*zeros, *w, bias=b.cuda(), act="relu", dtype=torch.float32, save=True)
    assert bool((ck_s[:, 0] >= 2.0 ** 121).all()) and torch.equal(y.cpu(), b.clamp(min=0).expand(M, N))
    dy = torch.ones((M, N), device="cuda")
    dz = qlin.qlin_act_bwd(dy, ck, ck_s, "relu", dtype=torch.float32)[0]
    assert torch.equal(dz.cpu(), (b > 0).float().expand(M, N))


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_a_block_with_an_infinity(act):
    """Its scale is not finite and its codes say nothing of the other 31 values: none of
    their gradients is a number, and the next block's are as without it."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("infinite block", act)
    M, N, K = 5, 64, 64
    zeros = torch.zeros((M, K), dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    b = torch.linspace(-2.0, 2.0, N, device="cuda")
    clean = qlin.qlin_fwd_act(*zeros, *w, bias=b, act=act, save=True)
    dy = torch.ones((M, N), device="cuda")
    want = qlin.qlin_act_bwd(dy, *clean[1:], act, dtype=torch.float32)[0]
    for bad in (float("inf"), -float("inf"), float("nan")):
        b[9] = bad
        y, ck, ck_s = qlin.qlin_fwd_act(*zeros, *w, bias=b, act=act, dtype=torch.float32, save=True)
        assert not ck_s[:, 0].isfinite().any()
        if bad != bad:
            assert y[:, 9].isnan().all()
        elif bad > 0:
            assert (y[:, 9] == bad).all()
        sw, sx = torch.ones(N, device="cuda"), torch.ones(M, device="cuda")
        dz, s1, s2, db = qlin.qlin_act_bwd(dy, ck, ck_s, act, sw=sw, sx=sx, dtype=torch.float32, want_db=True)
        assert dz[:, :32].isnan().all() and torch.equal(dz[:, 32:], want[:, 32:])
        assert not s1.isfinite().any() and not s2[:32].isfinite().any() and not db[:32].isfinite().any()
        assert s2[32:].isfinite().all() and db[32:].isfinite().all()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_an_infinite_scale(act):
    """Of a checkpoint from elsewhere: the same, whatever its codes."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("infinite scale", act)
    ck = torch.arange(-64, 64, dtype=torch.int8, device="cuda").view(2, 64)
    ck_s = torch.ones((2, 2), device="cuda")
    ck_s[:, 0] = float("inf")
    dz = qlin.qlin_act_bwd(torch.ones((2, 64), device="cuda"), ck, ck_s, act, dtype=torch.float32)[0]
    assert dz[:, :32].isnan().all() and dz[:, 32:].isfinite().all()
