"""Layer norm on rows whose strides say little."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_rows_of_one_element_in_any_stride(cuda_lib):
    """A row of one element is contiguous whatever the stride of its last dimension; rows must still not overlap."""
    x = torch.randn(240, device="cuda")
    column = x.as_strided((20, 1), (12, 5))
    assert not column.is_contiguous()
    b = torch.tensor([0.5], device="cuda")
    y, mean, rstd = cuda_lib.layer_norm(column, None, b, stats=True)
    assert torch.equal(y, torch.full((20, 1), 0.5, device="cuda")) and torch.equal(mean, column[:, 0])
    dx, dw, db = cuda_lib.layer_norm_backward(column, column, mean, rstd)
    assert not dx.any() and not dw.any()
    assert abs(float(db) - float(column.double().sum())) < 1e-4
    with pytest.raises(ValueError):
        cuda_lib.layer_norm(x.as_strided((20, 1), (0, 5)))
