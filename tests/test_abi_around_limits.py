"""Sizes that the launches around the projection cannot hold are refused before
anything is launched (fake addresses: only where no GPU is present)."""
import pytest

from tests.test_abi import P, L, _cpu_only  # noqa: F401
from tests.test_abi_around import _bwd

WIDE = dict(dx=None, qg1=None, sg1=None, qw=None, M=0, L=1, ws_bytes=1 << 62)


@pytest.mark.parametrize("K,N,R", [(1 << 30, 64, 16), (1 << 27, 64, 128), (1 << 29, 16, 8)])
def test_adapter_bwd_refuses_gradients_past_a_launch(L, K, N, R):        # noqa: F811
    """A gradient's sums take a thread per four values, the preparation one workgroup
    per 32 x 32 of a matrix."""
    _cpu_only()
    assert L.qlin_adapter_bwd(*_bwd(**WIDE, K=K, N=N, R=R)) == 2
    assert L.qlin_adapter_bwd_ws_bytes(0, N, K, 1, R) == 0


def test_adapter_bwd_workspace_at_the_limit(L):        # noqa: F811
    assert L.qlin_adapter_bwd_ws_bytes(0, 64, (1 << 29) - 576, 1, 32) > 0
    assert L.qlin_adapter_bwd_ws_bytes(0, 64, (1 << 29) - 560, 1, 32) == 0


@pytest.mark.parametrize("N,K", [(1 << 24, 16), ((1 << 24) + 5, 16384), (1 << 22, 16400), (1 << 30, 32)])
def test_updates_refuse_rows_past_a_launch(L, N, K):        # noqa: F811
    """A row takes 256 threads, above 16384 columns 1024."""
    _cpu_only()
    A, B, C, D, E = (P + (1 << 44) * k for k in range(1, 6))
    assert L.qlin_sgd_requant(A, B, C, N, K, 0.1, 0, 0, None, None, None) == 2
    assert L.qlin_adamw_requant(A, B, C, D, E, N, K, 0.1, 0.9, 0.99, 1e-8, 0.0, 0, 1, *[None] * 4, None) == 2
    assert L.qlin_wn_sgd_requant(A, B, C, D, E, N, K, 0.1, 0, 0, None, None, None) == 2


def test_weight_norm_preparation_refuses_rows_past_a_launch(L):      # noqa: F811
    _cpu_only()
    A, B, C, D = (P + (1 << 44) * k for k in range(1, 5))
    assert L.qlin_wn_init(A, B, 1 << 24, 32768, C, D, None) == 2
