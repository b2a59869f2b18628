"""The binding's compiled half, where no GPU is needed."""
import pytest
import torch


def _marshal():
    from w8a8_integer_linear_amd import _native
    _native._load_compiled()
    from w8a8_integer_linear_amd import _marshal
    return _marshal


def test_empty_has_the_type_and_shape_that_are_asked_for():
    m = _marshal()
    like = torch.nn.Parameter(torch.zeros(3))
    for dtype, shape in ((torch.int8, (2, 5)), (torch.bfloat16, (0, 7)), (torch.float32, (4,)),
                         (torch.uint8, ()), (torch.int32, (1, 2, 3, 4))):
        t = m.empty(like, dtype, *shape)
        assert t.dtype == dtype and t.shape == shape and t.device == like.device
        assert t.is_contiguous() and not t.requires_grad


@pytest.mark.parametrize("args,error", [
    ((), TypeError), ((torch.zeros(1),), TypeError), ((1, torch.int8, 2), TypeError),
    ((torch.zeros(1), 3, 2), TypeError), ((torch.zeros(1), torch.int8, "2"), TypeError),
    ((torch.zeros(1), torch.int8, 1, 1, 1, 1, 1), TypeError), ((torch.zeros(1), torch.int8, -2), RuntimeError),
    ((torch.zeros(1), torch.int8, 1 << 80), OverflowError), ((torch.zeros(1), torch.int8, 1 << 62), RuntimeError),
])
def test_empty_refuses(args, error):
    with pytest.raises(error):
        _marshal().empty(*args)
