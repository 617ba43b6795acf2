"""The counters of a ragged batch as lists (no GPU)."""
import pytest
import torch

import bit_asymmetric_kv_quantize_b200 as kivi


@pytest.mark.parametrize("B", [1, 2, 3])
def test_ragged_lengths_of_any_batch(B):
    st = torch.zeros(B, 2, dtype=torch.int64)
    st[:, 0] = 128 * torch.arange(1, B + 1)
    st.view(torch.int32).view(B, 4)[:, 2] = torch.arange(B, dtype=torch.int32) + 7
    st.view(torch.int32).view(B, 4)[B - 1, 3] = 1
    n_q, r, status = kivi.ragged_lengths(st.view(torch.uint8).view(-1))
    assert n_q == [128 * (b + 1) for b in range(B)] and r == [7 + b for b in range(B)]
    assert status == [0] * (B - 1) + [1]
