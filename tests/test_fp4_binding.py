"""The 4-bit operators' Python classes where no launch is needed (CPU)."""
import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib, api
from tests.test_fp4_host import lib  # noqa: F401  (a fixture)


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


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


@pytest.mark.parametrize("kind", ["Fp4PFFN", "Fp4MoE", "Fp8PFFN"])
def test_an_ffn_keeps_the_sizes_of_a_bounded_number_of_batches(kind, monkeypatch, lib):  # noqa: F811
    """A serving process sees any number of batch sizes; the workspace of each is what the library says."""
    monkeypatch.setattr(api, "_fp8_device", lambda *indices: indices[0])
    T, E, D, F = 2, 3, 64, 96
    lead = (T, E) if kind == "Fp4MoE" else (T,)
    if kind == "Fp8PFFN":
        w1, w2 = (api.Fp8Tensor(u8(T, k, n + -n % 16).view(torch.float8_e4m3fn), u8(T, 1, 4), n) for k, n in ((D, F), (F, D)))
        args, ask = (_lib.RM_FP8_SERVE,), _lib.rm_fp8_pffn_workspace
    else:
        w1, w2 = (api.Fp4Tensor(u8(*lead, n, 16 * (k // 32)), u8(*lead, 1, 2, 512), k, weight=True) for k, n in ((D, F), (F, D)))
        args, ask = (), getattr(_lib, {"Fp4PFFN": "rm_fp4_pffn_workspace", "Fp4MoE": "rm_fp4_moe_workspace"}[kind])
    f = getattr(api, kind)(w1, torch.zeros(*lead, F), w2, torch.zeros(*lead, D))
    for B in list(range(1, 300)) + [7, 299, 1]:
        work, n = f._work(B, *args, torch.device("cpu"))
        assert n == ask(f.c, B, *args) and work.numel() == n
    assert f._bytes.cache_info().currsize <= 64
