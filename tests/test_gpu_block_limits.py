"""The operators inside a feed-forward block past 32-bit byte offsets, in outputs and in
the weight, and past the rows that one launch holds.  Rows (outputs) do not depend on
one another, so the last ones are compared with those of a small call."""
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def _codes(torch, *shape):
    return torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda")


@pytest.mark.parametrize("gated", [False, True])
def test_outputs_past_4_gib(gated):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    torch.manual_seed(3)
    M, N, K, tail = 70000, 65536, 32, 300
    F = N // 2 if gated else N
    first = qlin.qlin_fwd_gated if gated else qlin.qlin_fwd_act
    qx, qw = _codes(torch, M, K), _codes(torch, N, K)
    sx, sw = torch.rand(M, device="cuda") + 0.5, (torch.rand(N, device="cuda") + 0.5) * 1e-4
    announce("outputs past 4 GiB", gated)
    y, ck, ck_s = first(qx, sx, qw, sw, act="silu", save=True)
    end = first(qx[-tail:].contiguous(), sx[-tail:].clone(), qw, sw, act="silu", save=True)
    assert y.numel() * y.element_size() > 1 << 32 and ck.numel() > 1 << 32
    for a, b in zip((y, ck, ck_s), end):
        assert torch.equal(a[-tail:], b)
    announce("their backward", gated)
    dz, s1, s2, db = qlin.qlin_act_bwd(y, ck, ck_s, "silu", gated=gated, sw=sw, sx=sx, want_db=True)
    want = qlin.qlin_act_bwd(end[0], end[1], end[2], "silu", gated=gated, sw=sw, sx=sx[-tail:].clone())
    assert torch.equal(dz[-tail:], want[0]) and torch.equal(s1[-tail:], want[1])
    half = M // 2
    parts = [qlin.qlin_act_bwd(y[r], ck[r], ck_s[r], "silu", gated=gated, sw=sw, sx=sx[r])[2]
             for r in (slice(0, half), slice(half, M))]
    assert torch.equal(s2, torch.maximum(*parts))
    some = dz[:, N - 64:].double()          # a bf16 rounding each, and fewer than 2^14 sums in a row
    assert ((some.sum(0) - db[N - 64:].double()).abs() <= some.abs().sum(0) * (2.0 ** -8 + 2.0 ** -9)).all()
    announce("its codes", gated)
    q1, q2 = qlin.qlin_quantize_grad_scaled(dz, sw, sx, s1, s2)
    e1, e2 = qlin.qlin_quantize_grad_scaled(dz[-tail:], sw, sx[-tail:].clone(), s1[-tail:].clone(), s2)
    assert torch.equal(q1[-tail:], e1) and torch.equal(q2[-tail:], e2)


@pytest.mark.parametrize("M", [3, 12, 40, 70])
def test_the_longest_weight(M):
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    torch.manual_seed(4)
    N, K, tail = 2097152, 2064, 4096
    qx, qw = _codes(torch, M, K), _codes(torch, N, K)
    sx, sw = torch.rand(M, device="cuda") + 0.5, (torch.rand(N, device="cuda") + 0.5) * 1e-5
    for save in (False, True):
        announce("weight past 4 GiB", M, save)
        y, ck, ck_s = qlin.qlin_fwd_act(qx, sx, qw, sw, act="gelu", save=save)
        end = qlin.qlin_fwd_act(qx, sx, qw[-tail:], sw[-tail:], act="gelu", save=save)
        assert torch.equal(y[:, -tail:], end[0])
        if save:
            assert torch.equal(ck[:, -tail:], end[1]) and torch.equal(ck_s[:, -tail // 32:], end[2])
        announce("gated weight past 4 GiB", M, save)
        F = N // 2
        y, ck, ck_s = qlin.qlin_fwd_gated(qx, sx, qw, sw, act="silu", save=save)
        two = torch.cat([qw[F - tail:F], qw[-tail:]]), torch.cat([sw[F - tail:F], sw[-tail:]])
        end = qlin.qlin_fwd_gated(qx, sx, *two, act="silu", save=save)
        assert torch.equal(y[:, -tail:], end[0])
        if save:
            assert torch.equal(ck[:, -tail:], end[1][:, tail:]) and torch.equal(ck_s[:, -tail // 32:],
                                                                               end[2][:, tail // 32:])


def test_more_rows_than_a_launch_of_scales_holds():
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    M, F, tail = (1 << 28) + 64, 16, 1000
    announce("backward of 2^28 rows")
    dy = torch.ones((M, F), dtype=torch.bfloat16, device="cuda")
    dy[-tail:] = torch.randn((tail, F), device="cuda")
    ck = torch.full((M, F), 64, dtype=torch.int8, device="cuda")
    ck_s = torch.full((M, 1), 0.5, device="cuda")
    sw = torch.rand(F, device="cuda") + 0.5
    dz, s1, _, _ = qlin.qlin_act_bwd(dy, ck, ck_s, "relu", sw=sw)
    end = qlin.qlin_act_bwd(dy[-tail:], ck[-tail:], ck_s[-tail:], "relu", sw=sw)
    assert torch.equal(dz[-tail:], end[0]) and torch.equal(s1[-tail:], end[1])
    rest = s1[:-tail]
    scale = torch.tensor(float(sw.max()) / 127)         # rounded once
    assert bool((rest == scale.cuda()).all()) and torch.equal(dz[:-tail:4099], dy[:-tail:4099])
