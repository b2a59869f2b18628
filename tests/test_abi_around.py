"""Refusals of the entry points around the projection (norm, adapters, AdamW over
many tensors): host checks, before anything is launched.

As in test_abi.py the addresses are fake and the tests run only where no GPU is
present."""
import ctypes

import pytest

from tests.test_abi import ODD, P, L, _cpu_only  # noqa: F401

BIG = 1 << 42        # distance between the fake arrays: none overlap
A = [P + BIG * k for k in range(1, 24)]


def _norm(**kw):
    a = dict(x=A[0], residual=A[1], dtype=1, rows=4, cols=256, gamma=A[2], eps=1e-6, had=0, h=A[3],
             q=A[4], s=A[5], rstd=A[6], y=A[7])
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), 1), (dict(x=ODD), 1), (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(cols=24), 1),
    (dict(cols=0), 1), (dict(gamma=None), 1), (dict(gamma=ODD), 1), (dict(eps=0.0), 1),
    (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(had=3), 1), (dict(had=512), 1), (dict(had=-2), 1), (dict(q=None), 1), (dict(s=None), 1),
    (dict(rstd=None), 1), (dict(y=ODD), 1), (dict(h=None), 1), (dict(residual=None), 1),
    (dict(h=A[0] + 16), 1),                 # a shifted copy of x
    (dict(q=A[0]), 1), (dict(y=A[1] + 64), 1), (dict(s=A[6]), 1), (dict(gamma=A[3]), 1),
    (dict(cols=131072 + 16), 2), (dict(rows=(1 << 30) + 1), 2),
    (dict(rows=0, x=None, residual=None, h=None, q=None, s=None, rstd=None, y=None), 0),
])
def test_rmsnorm_quant_refusals(L, kw, expect):        # noqa: F811
    _cpu_only()
    assert L.qlin_rmsnorm_quant(*_norm(**kw)) == expect


def _norm_bwd(**kw):
    a = dict(dn=A[0], dn_dtype=0, h=A[1], dres=A[2], dtype=1, rstd=A[3], gamma=A[4], rows=4, cols=256,
             dh=A[5], dgamma=A[6], ws=A[7], ws_bytes=1 << 20)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dn=None), 1), (dict(dn_dtype=3), 1), (dict(dtype=-1), 1), (dict(h=ODD), 1),
    (dict(rstd=None), 1), (dict(gamma=None), 1), (dict(dh=None), 1), (dict(dgamma=None), 1),
    (dict(ws=None), 1), (dict(ws_bytes=16), 1), (dict(cols=40), 1), (dict(rows=-2), 1),
    (dict(dh=A[1]), 1), (dict(dh=A[2] + 16), 1), (dict(ws=A[0] + 32), 1), (dict(dgamma=A[4]), 1),
    (dict(cols=1 << 20), 2),
])
def test_rmsnorm_bwd_refusals(L, kw, expect):          # noqa: F811
    _cpu_only()
    assert L.qlin_rmsnorm_bwd(*_norm_bwd(**kw)) == expect


def _fwd(**kw):
    a = dict(qx=A[0], sx=A[1], qw=A[2], sw=A[3], bias=A[4], a=A[5], b=A[6], w_dtype=1, scale=A[7],
             ids=A[8], M=20, N=64, K=64, L=3, R=16, u=A[9], y=A[10], ws=A[11], ws_bytes=1 << 31)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(qx=None), 1), (dict(sx=None), 1), (dict(qw=ODD), 1), (dict(sw=None), 1), (dict(bias=ODD), 1),
    (dict(a=None), 1), (dict(b=None), 1), (dict(w_dtype=2), 1), (dict(scale=None), 1),
    (dict(ids=None), 1), (dict(ids=ODD), 1), (dict(M=-1), 1), (dict(N=40), 1), (dict(K=8), 1),
    (dict(L=0), 1), (dict(R=0), 1), (dict(R=12), 1), (dict(R=136), 1), (dict(u=None), 1),
    (dict(y=None), 1), (dict(y=A[4]), 1), (dict(u=A[8]), 1), (dict(y=A[9]), 1),
    (dict(K=131088), 2), (dict(M=1048561), 2), (dict(L=1 << 40), 2), (dict(K=131056, L=1 << 30), 2),
    (dict(M=0, qx=None, sx=None, sw=None, ids=None, u=None, y=None, ws=None, ws_bytes=0), 0),
])
def test_adapter_fwd_refusals(L, kw, expect):          # noqa: F811
    _cpu_only()
    assert L.qlin_adapter_fwd(*_fwd(**kw)) == expect


def test_adapter_fwd_needs_its_workspace(L):           # noqa: F811
    _cpu_only()
    big = dict(M=600, N=7168, K=5376)
    need = L.qlin_adapter_fwd_ws_bytes(600, 7168, 5376, 3, 16)
    assert need > 0
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=ODD), dict(ws=A[10] + 4096)):
        assert L.qlin_adapter_fwd(*_fwd(**big, **kw)) == 1


def _bwd(**kw):
    a = dict(dy=A[0], dy_dtype=1, qg1=A[1], sg1=A[2], qw=A[3], qx=A[4], sx=A[5], u=A[6], a=A[7],
             b=A[8], w_dtype=0, scale=A[9], ids=A[10], order=A[11], start=A[12], M=20, N=64, K=128,
             L=3, R=16, had=64, dx=A[13], da=A[14], db=A[15], ws=A[16], ws_bytes=1 << 31)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), 1), (dict(dy_dtype=7), 1), (dict(qg1=None), 1), (dict(sg1=None), 1),
    (dict(qw=None), 1), (dict(qx=None), 1), (dict(sx=ODD), 1), (dict(u=None), 1), (dict(a=ODD), 1),
    (dict(b=None), 1), (dict(scale=None), 1), (dict(ids=None), 1), (dict(order=None), 1),
    (dict(start=None), 1), (dict(R=20), 1), (dict(L=0), 1), (dict(had=48), 1), (dict(had=256), 1),
    (dict(da=None), 1), (dict(db=None), 1), (dict(ws=None), 1), (dict(ws_bytes=0), 1),
    (dict(da=A[15]), 1), (dict(dx=A[0]), 1), (dict(db=A[12]), 1), (dict(ws=A[14] + 256), 1),
    (dict(N=131088), 2), (dict(L=1024), 2), (dict(M=1048561), 2),
    (dict(dx=None, qg1=None, sg1=None, qw=None, N=131088), 2),
])
def test_adapter_bwd_refusals(L, kw, expect):          # noqa: F811
    _cpu_only()
    assert L.qlin_adapter_bwd(*_bwd(**kw)) == expect


@pytest.mark.parametrize("args,expect", [
    ((None, 4, 3, A[0], A[1]), 1), ((A[2], 4, 3, None, A[1]), 1), ((A[2], 4, 3, A[0], None), 1),
    ((A[2], -1, 3, A[0], A[1]), 1), ((A[2], 4, 0, A[0], A[1]), 1), ((ODD, 4, 3, A[0], A[1]), 1),
    ((A[2], 4, 3, A[2], A[1]), 1), ((A[2], 4, 1024, A[0], A[1]), 2), ((A[2], 1 << 21, 3, A[0], A[1]), 2),
])
def test_adapter_group_refusals(L, args, expect):      # noqa: F811
    _cpu_only()
    assert L.qlin_adapter_group(*args, None) == expect


def _desc(**kw):
    from w8a8_integer_linear_amd._native import TensorDesc
    a = dict(p=A[0], g=A[1], m=A[2], v=A[3], m_scale=None, v_scale=None, numel=1000, index0=0,
             weight_decay=0.0, p_dtype=0, g_dtype=1, state_bits=32)
    a.update(kw)
    return TensorDesc(**a)


def _plan(L, *descs, room=1 << 20):                    # noqa: F811
    from w8a8_integer_linear_amd._native import TensorDesc
    arr = (TensorDesc * max(1, len(descs)))(*descs)
    buf = ctypes.create_string_buffer(room)
    return L.qlin_adamw_tensors_plan(arr, len(descs), ctypes.addressof(buf), room), arr, buf


EIGHT = dict(state_bits=8, m_scale=A[4], v_scale=A[5])


@pytest.mark.parametrize("kw,expect", [
    (dict(), 0), (EIGHT, 0), (dict(numel=0, p=None, g=None, m=None, v=None), 0),
    (dict(p=None), 1), (dict(g=ODD), 1), (dict(m=None), 1), (dict(v=ODD), 1), (dict(numel=-1), 1),
    (dict(p_dtype=2), 1), (dict(g_dtype=-1), 1), (dict(state_bits=16), 1), (dict(index0=4), 1),
    (dict(index0=-8), 1), (dict(weight_decay=-0.1), 1), (dict(weight_decay=float("nan")), 1),
    (dict(m_scale=A[4]), 1), (dict(EIGHT, v_scale=None), 1), (dict(EIGHT, m_scale=A[4] + 2), 1),
    (dict(EIGHT, m_scale=A[3] + 4), 1), (dict(v=A[2] + 1024), 1), (dict(p=A[1] + 16), 1),
    (dict(numel=1 << 43), 2),
])
def test_plan_refusals(L, kw, expect):                 # noqa: F811
    assert _plan(L, _desc(**kw))[0] == expect


def test_plan_of_several(L):                           # noqa: F811
    two = _desc(p=A[6], g=A[1], m=A[7], v=A[8], numel=9000)         # one gradient may serve two
    st, arr, buf = _plan(L, _desc(), two)
    assert st == 0
    assert L.qlin_adamw_tensors_chunks(arr, 2) == 1 + 3
    assert L.qlin_adamw_tensors_plan_bytes(arr, 2) == 2 * 80 + 4 * 4
    assert list((ctypes.c_int32 * 4).from_buffer(buf, 160)) == [0, 1, 1, 1]
    assert _plan(L, _desc(), _desc())[0] == 1                       # the same tensor twice
    assert _plan(L, _desc(), _desc(p=A[6], m=A[7], v=A[8], g=A[2]))[0] == 1
    assert _plan(L, _desc(), two, room=100)[0] == 1
    assert _plan(L)[0] == 0
    assert L.qlin_adamw_tensors_plan(None, 1, None, 0) == 1


@pytest.mark.parametrize("args,expect", [
    ((None, 1, 4, 1e-3, 0.9, 0.999, 1e-8, 0, 1), 1), ((ODD, 1, 4, 1e-3, 0.9, 0.999, 1e-8, 0, 1), 1),
    ((P, 0, 4, 1e-3, 0.9, 0.999, 1e-8, 0, 1), 1), ((P, 1, -4, 1e-3, 0.9, 0.999, 1e-8, 0, 1), 1),
    ((P, 1, 4, float("inf"), 0.9, 0.999, 1e-8, 0, 1), 1), ((P, 1, 4, 1e-3, 1.0, 0.999, 1e-8, 0, 1), 1),
    ((P, 1, 4, 1e-3, 0.9, -0.1, 1e-8, 0, 1), 1), ((P, 1, 4, 1e-3, 0.9, 0.999, 0.0, 0, 1), 1),
    ((P, 1, 4, 1e-3, 0.9, 0.999, 1e-60, 0, 1), 1), ((P, 1, 4, 1e-3, 0.9, 0.999, 1e-8, 0, 0), 1),
    ((P, 1, 1 << 40, 1e-3, 0.9, 0.999, 1e-8, 0, 1), 2), ((P, 1, 4, 1e-3, 0.9, 0.999, 1e-8, 0, 1 << 63), 2),
    ((None, 0, 0, 1e-3, 0.9, 0.999, 1e-8, 0, 1), 0),
])
def test_adamw_tensors_refusals(L, args, expect):      # noqa: F811
    _cpu_only()
    assert L.qlin_adamw_tensors(*args, None) == expect


def test_workspace_sizes_of_refused_shapes(L):         # noqa: F811
    assert L.qlin_rmsnorm_bwd_ws_bytes(4, 24) == 0 and L.qlin_rmsnorm_bwd_ws_bytes(-1, 32) == 0
    assert L.qlin_rmsnorm_bwd_ws_bytes(4, 1 << 30) == 0
    for bad in ((1, 24, 64, 1, 8), (1, 64, 64, 0, 8), (1, 64, 64, 1, 9), (-1, 64, 64, 1, 8),
                (1 << 62, 64, 64, 1, 8), (1, 1 << 62, 64, 1, 8)):
        assert L.qlin_adapter_fwd_ws_bytes(*bad) == 0
        assert L.qlin_adapter_bwd_ws_bytes(*bad) == 0


def test_binding_refuses_host_and_strided_tensors():
    import torch

    import w8a8_integer_linear_amd as qlin
    t = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        qlin.qlin_rmsnorm_quant(t, torch.ones(64), 1e-6)
    with pytest.raises(ValueError):
        qlin.qlin_rmsnorm_bwd(t, t, torch.ones(4), torch.ones(64))
    with pytest.raises(ValueError):
        qlin.qlin_adapter_group(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        qlin.qlin_adamw_tensors_plan([dict(p=t, g=t, m=t, v=t)])
