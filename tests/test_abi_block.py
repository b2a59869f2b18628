"""Refusals of the entry points inside a feed-forward block: host checks, before
anything is launched.  As in test_abi.py the addresses are fake and the tests run only
where no GPU is present."""
import pytest

from tests.test_abi import ODD, P, L, _cpu_only  # noqa: F401

A = [P + (1 << 42) * k for k in range(1, 16)]       # none overlap


def _act(**kw):
    a = dict(qx=A[0], sx=A[1], qw=A[2], sw=A[3], bias=A[4], act=3, residual=A[5], res_dtype=1, M=20, N=64,
             K=64, y=A[6], y_dtype=1, ck=A[7], ck_s=A[8], ws=A[9], ws_bytes=1 << 31)
    a.update(kw)
    return (*a.values(), None)


NOTHING = dict(qx=None, sx=None, sw=None, y=None, ck=None, ck_s=None, ws=None, ws_bytes=0, M=0)


@pytest.mark.parametrize("kw,expect", [
    (dict(qx=None), 1), (dict(qx=ODD), 1), (dict(sx=None), 1), (dict(sx=ODD), 1), (dict(qw=None), 1),
    (dict(sw=None), 1), (dict(bias=ODD), 1), (dict(act=5), 1), (dict(act=-1), 1), (dict(residual=ODD), 1),
    (dict(res_dtype=2), 1), (dict(M=-1), 1), (dict(N=40), 1), (dict(N=0), 1), (dict(K=8), 1),
    (dict(y=None), 1), (dict(y=ODD), 1), (dict(y_dtype=7), 1), (dict(ck=None), 1), (dict(ck_s=None), 1),
    (dict(ck=ODD), 1), (dict(ck_s=ODD), 1), (dict(y=A[0]), 1), (dict(ck=A[2] + 64), 1), (dict(ck_s=A[1]), 1),
    (dict(ck=A[6]), 1), (dict(y=A[4]), 1),
    (dict(residual=A[6], res_dtype=0), 1),          # y itself, but of another type
    (dict(residual=A[6] + 64), 1), (dict(ck=A[5]), 1),
    (dict(K=131088), 2), (dict(N=2097168), 2), (dict(N=1 << 40), 2), (dict(M=(1 << 30) + 1), 2),
    (dict(residual=None, res_dtype=9, **NOTHING), 0), (dict(bias=None, residual=None, **NOTHING), 0),
])
def test_act_refusals(L, kw, expect):        # noqa: F811
    _cpu_only()
    assert L.qlin_fwd_act(*_act(**kw)) == expect


def _gated(**kw):
    a = dict(qx=A[0], sx=A[1], qw=A[2], sw=A[3], bias=A[4], act=2, M=20, F=64, K=64, y=A[6], y_dtype=0,
             ck=A[7], ck_s=A[8], ws=A[9], ws_bytes=1 << 31)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(qx=None), 1), (dict(sw=None), 1), (dict(act=9), 1), (dict(F=24), 1), (dict(F=0), 1), (dict(F=-16), 1),
    (dict(K=40), 1), (dict(M=-3), 1), (dict(y_dtype=-1), 1), (dict(y=A[1]), 1), (dict(ck=None), 1),
    (dict(y=A[2] + 64 * 64), 1),                    # over the second half's rows
    (dict(ck_s=A[7] + 20 * 64), 1),                 # over the second half's codes
    (dict(F=1048592), 2), (dict(F=1 << 61), 2), (dict(F=(1 << 63) - 16), 2), (dict(K=131088), 2),
    (NOTHING, 0),
])
def test_gated_refusals(L, kw, expect):      # noqa: F811
    _cpu_only()
    assert L.qlin_fwd_gated(*_gated(**kw)) == expect


def test_forward_needs_its_workspace(L):     # noqa: F811
    _cpu_only()
    need = L.qlin_fwd_act_ws_bytes(600, 7168, 5376)
    assert need > 0 and need == L.qlin_fwd_gated_ws_bytes(600, 3584, 5376)
    assert need == L.qlin_product_ws_bytes(0, 600, 7168, 5376)
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=ODD), dict(ws=A[6] + 4096)):
        assert L.qlin_fwd_act(*_act(M=600, N=7168, K=5376, **kw)) == 1
        assert L.qlin_fwd_gated(*_gated(M=600, F=3584, K=5376, **kw)) == 1
    assert L.qlin_fwd_act_ws_bytes(600, 7168, 131088) == 0
    for bad in (-1, 1 << 62, (1 << 63) - 1):
        assert L.qlin_fwd_gated_ws_bytes(600, bad, 64) == 0


def test_calls_that_split_nothing_need_no_workspace(L):      # noqa: F811
    for M, N, K in ((1, 28672, 4096), (16, 4096, 14336), (64, 28672, 4096), (128, 4096, 14336), (512, 2048, 5376),
                    (0, 64, 64)):
        assert L.qlin_fwd_act_ws_bytes(M, N, K) == 0 and L.qlin_fwd_gated_ws_bytes(M, N // 2, K) == 0
    _cpu_only()
    none = dict(ws=None, ws_bytes=0)
    assert L.qlin_fwd_act(*_act(M=600, N=7168, K=5376, **none)) == 1


def _bwd(**kw):
    a = dict(dy=A[0], dy_dtype=0, ck=A[1], ck_s=A[2], act=2, gated=1, sw=A[3], sx=A[4], M=20, F=64, dz=A[5],
             dz_dtype=1, s1=A[6], s2=A[7], db=A[8], ws=A[9], ws_bytes=1 << 31)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), 1), (dict(dy=ODD), 1), (dict(dy_dtype=2), 1), (dict(ck=None), 1), (dict(ck=ODD), 1),
    (dict(ck_s=None), 1), (dict(act=5), 1), (dict(gated=2), 1), (dict(gated=-1), 1), (dict(sw=None), 1),
    (dict(s1=None), 1), (dict(sx=None), 1), (dict(s2=None), 1), (dict(sw=ODD), 1), (dict(s2=ODD), 1),
    (dict(db=ODD), 1), (dict(M=-1), 1), (dict(F=20), 1), (dict(F=0), 1), (dict(dz=None), 1), (dict(dz=ODD), 1),
    (dict(dz_dtype=5), 1), (dict(ws=None), 1), (dict(ws_bytes=64), 1), (dict(ws=ODD), 1),
    (dict(dz=A[0]), 1), (dict(dz=A[1]), 1), (dict(s1=A[4]), 1), (dict(s2=A[8]), 1), (dict(ws=A[5] + 256), 1),
    (dict(db=A[2]), 1), (dict(dz=A[1] - 16 * 16), 1),
    (dict(F=1048592), 2), (dict(F=2097168, gated=0), 2), (dict(M=(1 << 30) + 1), 2), (dict(F=1 << 62), 2),
])
def test_act_bwd_refusals(L, kw, expect):    # noqa: F811
    _cpu_only()
    assert L.qlin_act_bwd(*_bwd(**kw)) == expect


def test_act_bwd_workspace_sizes(L):         # noqa: F811
    assert L.qlin_act_bwd_ws_bytes(0, 64, 0) == 0
    # A row maximum per token and window, two values per column and row group.
    assert L.qlin_act_bwd_ws_bytes(20, 64, 1) >= 4 * (20 + 2 * 128)
    for bad in ((-1, 64, 0), (4, 24, 0), (4, 1048592, 1), (1 << 40, 64, 0), (4, -16, 1)):
        assert L.qlin_act_bwd_ws_bytes(*bad) == 0


def _codes(**kw):
    a = dict(dy=A[0], dtype=1, M=20, N=64, sw=A[1], sx=A[2], s1=A[3], s2=A[4], q1=A[5], q2=A[6])
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    *[({k: v}, 1) for k in ("dy", "sw", "sx", "s1", "s2", "q1", "q2") for v in (None, ODD)],
    (dict(dtype=3), 1), (dict(M=-1), 1), (dict(N=24), 1), (dict(q1=A[6]), 1), (dict(q2=A[0] + 64), 1),
    (dict(q1=A[3] - 16), 1), (dict(N=131088), 2), (dict(M=65535 * 16 + 1), 2),
    (dict(dy=None, sw=None, sx=None, s1=None, s2=None, q1=None, q2=None, M=0), 0),
])
def test_codes_refusals(L, kw, expect):      # noqa: F811
    _cpu_only()
    assert L.qlin_quantize_grad_scaled(*_codes(**kw)) == expect


def test_binding_refuses_host_tensors_and_unknown_names():
    import torch

    import w8a8_integer_linear_amd as qlin
    q, f = torch.zeros((4, 64), dtype=torch.int8), torch.ones(4)
    w = torch.zeros((32, 64), dtype=torch.int8), torch.ones(32)
    for first in (qlin.qlin_fwd_act, qlin.qlin_fwd_gated):
        with pytest.raises(ValueError, match="GPU"):
            first(q, f, *w)
        with pytest.raises(ValueError, match="act is one of"):
            first(q, f, *w, act="swish")
    with pytest.raises(ValueError, match="as many others"):
        qlin.qlin_fwd_gated(q, f, w[0][:31], w[1][:31])
    with pytest.raises(ValueError, match="GPU"):
        qlin.qlin_act_bwd(torch.zeros((4, 32)), q[:, :32].contiguous(), f, "silu")
    with pytest.raises(ValueError, match="GPU"):
        qlin.qlin_quantize_grad_scaled(torch.zeros((4, 32)), w[1], f, f, w[1])
