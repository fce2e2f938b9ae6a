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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_bias_is_kept_aligned(dtype):
    """Views into a larger buffer among them; a float32 bias that is as it has to be is kept itself."""
    flat = torch.arange(64, dtype=dtype)
    for at in range(9):
        b = flat[at:at + 48].view(3, 16)
        kept = api._kept_bias(b)
        assert kept.dtype == torch.float32 and kept.is_contiguous() and kept.data_ptr() % 16 == 0 and torch.equal(kept, b.float())
        assert (kept.data_ptr() == b.data_ptr()) == (dtype == torch.float32 and b.data_ptr() % 16 == 0)
    kept = api._kept_bias(flat[:48].view(16, 3).T)
    assert kept.is_contiguous() and torch.equal(kept, flat[:48].view(16, 3).T.float())
