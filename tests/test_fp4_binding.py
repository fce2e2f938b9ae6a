"""The 4-bit operators' Python classes where no launch is needed (CPU)."""
import pytest
import torch

from rankmixer_feature_interaction_gb300 import api


@pytest.mark.parametrize("cols", [1, 40, 512, 600])
def test_a_tensor_of_no_rows_has_codes_and_scales(cols):
    """As expert_gather to 4 bits gives where there is room for no row."""
    q = api._fp4_new((0,), cols, False, torch.device("cpu"), -1)
    nb = -(-cols // 32)
    assert q.shape == (0, cols) and q.nbytes == 0
    assert q.codes.shape == (0, 16 * nb) and q.scales.shape == (0, -(-nb // 16) * 16)
    assert q.codes.dtype is torch.uint8 and q.scales.dtype is torch.uint8
    again = api.Fp4Tensor(q.codes, q.scales, cols)
    assert again.shape == q.shape and again.codes is q.codes
