"""fp32 operands of the adapters' products are held to their 24 bits: inputs whose
results are single products, so that nothing but the operands' splits and a few
roundings can show.

An fp32 value is three bf16 terms exactly (8 + 8 + 8 bits, each the rounded rest of
the ones before, at most 2^-8 of it), so a product with a one-term operand is the
sum of three exact partial products, and one of two split operands lacks the three
partial products below: |t1 t2| + |t2 t1| + |t2 t2| <= (2 * 2^-24 + 2^-32) (1 + 2^-7).
The rest is at most six additions of exact partial products, each of a result no
larger than (1 + 2^-7) of the product and within 2^-23 of it (rounded or cut off):
    ONE = 6 * 2^-23 (1 + 2^-7) + 2.1 * 2^-24 < 2^-20
of the product.  With two terms, or without any one of the six partial products, the
error reaches 2^-17 (the first test)."""
import pytest
import torch as cpu

from tests import test_gpu_adapter as plain
from tests.gpu_util import announce, torch_cuda

ONE = 2.0 ** -20
U = 2.0 ** -24


def _full(shape, g):
    """fp32 values whose 24 bits are all in use, of sizes from 2^-4 to 2^4."""
    k = cpu.randint(0, 1 << 22, shape, generator=g) * 2 + 1
    e = cpu.randint(-4, 4, shape, generator=g)
    sign = cpu.randint(0, 2, shape, generator=g) * 2 - 1
    return (sign * (1 + k * 2.0 ** -23) * 2.0 ** e.double()).float()


def _terms(x):
    rest, out = x.clone(), []
    for _ in range(3):
        out.append(rest.to(cpu.bfloat16).float())
        rest = rest - out[-1]
    assert (rest == 0).all()
    return [t.double() for t in out]


def test_the_bound_tells_three_terms_from_two():
    g = cpu.Generator().manual_seed(1)
    x, w = _full((20_000,), g), _full((20_000,), g)
    p, q = _terms(x), _terms(w)
    exact = x.double() * w.double()
    pairs = [(i, j) for i in range(3) for j in range(3) if i + j <= 2]

    def worst(used):
        return ((sum(p[i] * q[j] for i, j in used) - exact).abs() / exact.abs()).max().item()

    assert worst(pairs) < 2.0 ** -22
    for left_out in pairs:
        assert worst([x for x in pairs if x != left_out]) > 4 * ONE
    assert worst([(i, j) for i, j in pairs if i < 2 and j < 2]) > 4 * ONE
    assert ((p[0] + p[1] - x.double()).abs() / x.double().abs()).max() > 4 * ONE


def _distinct(n, most, g):
    """n places below most, distinct where there are enough."""
    return cpu.cat([cpu.randperm(most, generator=g) for _ in range(-(-n // most))])[:n]


# (weight streaming; a wave per token and rank; the tiled product with the term apart;
# the term in the products' epilogues)
FWD = [(7, 256, 512, 3, 16), (16, 64, 4112, 2, 128), (40, 272, 512, 3, 24), (300, 528, 272, 4, 40),
       (611, 1024, 2048, 8, 32), (2100, 4112, 96, 5, 24), (4500, 2064, 64, 2, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,L,R", FWD)
@pytest.mark.parametrize("w", ["f32", "bf16"])
def test_forward_of_single_products(M, N, K, L, R, w):
    """A token's only code is a 1 in column k, whose only rank is k % R: u is A's
    value times the factor, rounded once, and y is that u times B's value."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("single products", M, N, K, L, R, w)
    g = torch.Generator().manual_seed(M + R)
    kind = torch.float32 if w == "f32" else torch.bfloat16
    ids = torch.randint(0, L, (M,), generator=g, dtype=torch.int32)
    col = torch.randint(0, K, (M,), generator=g)
    qx = torch.zeros((M, K), dtype=torch.int8)
    qx[torch.arange(M), col] = 1
    a = _full((L, R, K), g)
    a *= (torch.arange(R)[:, None] == torch.arange(K) % R)
    a, b, scale = a.to(kind), _full((L, N, R), g).to(kind), _full((L,), g)
    y, u = qlin.qlin_adapter_fwd(qx.cuda(), torch.ones(M).cuda(), torch.zeros((N, K), dtype=torch.int8).cuda(),
                                 torch.ones(N).cuda(), a.cuda(), b.cuda(), scale.cuda(), ids.cuda())
    y, u = y.cpu(), u.cpu()
    l = ids.long()
    assert torch.equal(u, a.float()[l, :, col] * scale[l][:, None])
    r = col % R
    want = u.double()[torch.arange(M), r][:, None] * b.double()[l, :, r]
    assert (want != 0).all() and ((y.double() - want).abs() <= ONE * want.abs()).all()


BWD = [(7, 64, 48, 2, 24), (33, 1040, 512, 4, 8), (333, 512, 512, 5, 64), (700, 1024, 720, 2, 128),
       (1300, 1312, 1328, 3, 16), (2100, 96, 4096, 3, 16), (4500, 64, 2064, 2, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,L,R", BWD)
@pytest.mark.parametrize("w,dy", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_backward_of_single_products(M, N, K, L, R, w, dy):
    """A token's only gradient is in column n, whose only rank is n % R, and its only
    code a 1 in column k: v, hence dA, is one product, dx one more, dB another."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("single products backward", M, N, K, L, R, w, dy)
    g = torch.Generator().manual_seed(M + R)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    ids = torch.randint(0, L, (M,), generator=g, dtype=torch.int32)
    n, k, t = _distinct(M, N, g), _distinct(M, K, g), torch.arange(M)
    qx = torch.zeros((M, K), dtype=torch.int8)
    qx[t, k] = 1
    grad = torch.zeros((M, N))
    grad[t, n] = _full((M,), g)
    grad = grad.to(kind[dy])
    a = _full((L, R, K), g).to(kind[w])
    b = _full((L, N, R), g)
    b *= (torch.arange(N)[:, None] % R == torch.arange(R))
    b, u = b.to(kind[w]), _full((M, R), g)
    idc = ids.cuda()
    order, start = qlin.qlin_adapter_group(idc, L)
    one = torch.ones(M).cuda()
    dx, da, db = qlin.qlin_adapter_bwd(
        grad.cuda(), torch.zeros((M, N), dtype=torch.int8).cuda(), one,
        torch.zeros((N, K), dtype=torch.int8).cuda(), qx.cuda(), one, u.cuda(), a.cuda(), b.cuda(),
        torch.ones(L).cuda(), idc, order, start)
    l, r = ids.long(), n % R
    v = grad.double()[t, n] * b.double()[l, n, r]
    want = v[:, None] * a.double()[l, r]
    assert (want != 0).all() and ((dx.double().cpu() - want).abs() <= (2 * ONE + U) * want.abs()).all()
    if M <= min(N, K):      # (a gradient's value is then one token's)
        da64 = torch.zeros((L, R, K), dtype=torch.float64)
        da64[l, r, k] = v
        assert ((da.double().cpu() - da64).abs() <= ONE * da64.abs()).all()
        db64 = torch.zeros((L, N, R), dtype=torch.float64)
        db64[l, n] = grad.double()[t, n][:, None] * u.double()
        assert ((db.double().cpu() - db64).abs() <= ONE * db64.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["f32", "bf16"])
def test_mixed_tokens_of_rank_128(w):
    """Every 16 tokens hold both adapters and some none, at the largest rank, in the
    product's own epilogue.  Bounds as for the smaller shapes, with ONE per split
    product in place of two terms' 2^-15."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, N, K, L, R = 4500, 2064, 64, 2, 128
    announce("mixed tokens", M, N, K, L, R, w)
    c = plain._case(torch, M, N, K, L, R, w, seed=9)
    y, u = plain._run_fwd(qlin, plain._cuda(c))
    x = c["qx"].double() * c["sx"].double()[:, None]
    y64 = (x @ c["qw"].double().T) * c["sw"].double()
    bsize = y64.abs() + c["bias"].double().abs()
    y64 += c["bias"].double()
    u64, usize = torch.zeros((M, R), dtype=torch.float64), torch.zeros((M, R), dtype=torch.float64)
    low = torch.zeros_like(y64)
    for l in range(L):
        at = torch.nonzero(c["ids"] == l)[:, 0]
        A, B, sc = c["a"][l].double(), c["b"][l].double(), c["scale"][l].double()
        u64[at], usize[at] = sc * (x[at] @ A.T), sc * (x[at].abs() @ A.abs().T)
        y64[at] += u64[at] @ B.T
        low[at] = usize[at] @ B.abs().T
    assert ((u.double().cpu() - u64).abs() <= usize * (ONE + (K + 32) * U)).all()
    bound = 6 * U * (bsize + low) + low * (2 * ONE + (K + R + 64) * U)
    assert ((y.double().cpu() - y64).abs() <= bound).all()
