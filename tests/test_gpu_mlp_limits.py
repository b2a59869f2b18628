"""Passes that a feed-forward layer refuses leave its gradients as they were."""
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def test_a_weight_too_long_to_train():
    """Forward passes of a gated block whose first weight has more than 131072 rows run;
    its gradient's rows would be too long for their quantization."""
    torch = torch_cuda()
    import w8a8_integer_linear_amd as qlin
    announce("mlp: long weight")
    torch.manual_seed(2)
    M, K, F, N = 4, 16, 65552, 16
    w1, w2 = torch.randn((2 * F, K), device="cuda"), torch.randn((N, F), device="cuda")
    b1, b2 = torch.randn(2 * F, device="cuda"), torch.randn(N, device="cuda")
    block = qlin.MLPW8A8Training(w1, w2, b1, b2, act="silu", gated=True, had_block=16)
    y = block.forward(torch.randn((M, K), device="cuda"))
    assert y.shape == (M, N) and bool(y.isfinite().all())
    held = [t for fc in (block.fc1, block.fc2) for t in (fc.dw, fc.db)]
    for t in held:
        t.fill_(7.0)
    with pytest.raises(ValueError, match="131104 rows"):
        block.backward(torch.randn((M, N), device="cuda"))
    assert all(bool((t == 7).all()) for t in held)
    # The longest that is trained.
    block = qlin.MLPW8A8Training(w1[:131072], w2[:, :65536].contiguous(), act="silu", gated=True, had_block=16)
    block.forward(torch.randn((M, K), device="cuda"))
    assert bool(block.backward(torch.randn((M, N), device="cuda")).isfinite().all())
    assert bool(block.fc1.dw.isfinite().all()) and bool(block.fc2.dw.isfinite().all())
