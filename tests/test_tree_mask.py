"""What tree_mask refuses (no GPU)."""
import pytest
import torch

import bit_asymmetric_kv_quantize_b200 as kivi


@pytest.mark.parametrize("parents", [torch.tensor([[-1.0, 0.0]]), torch.tensor([[-0.5]]),
                                     torch.tensor([[False, False]])])
def test_parents_are_whole_numbers(parents):
    with pytest.raises(ValueError, match="int"):
        kivi.tree_mask(parents)


@pytest.mark.parametrize("shape", [(0, 3), (2, 0), (0, 0)])
def test_trees_have_nodes(shape):
    with pytest.raises(ValueError, match="shape"):
        kivi.tree_mask(torch.zeros(shape, dtype=torch.int64))


@pytest.mark.parametrize("dtype", [torch.int8, torch.int16, torch.int32, torch.int64])
def test_any_type_of_whole_numbers(dtype):
    m = kivi.tree_mask(torch.tensor([[-1, 0, 1], [-1, -1, 0]], dtype=dtype))
    assert m.dtype == torch.int32 and m.tolist() == [[[1], [3], [7]], [[1], [2], [5]]]
