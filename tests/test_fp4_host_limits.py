"""Host-side limits of the 4-bit operators and of the experts' rows (no GPU needed)."""
import ctypes

import pytest

from rankmixer_feature_interaction_gb300 import _lib
from tests.test_fp4_host import OK, lib, mem, wt  # noqa: F401  (fixtures)


@pytest.mark.parametrize("B", [1, 21, 22, 1024, 100000])
def test_moe_workspace_holds_every_experts_output_in_float32(lib, mem, B):  # noqa: F811
    """T = 32, E = 8, D = 1536, F = 2048: B = 22 is the first batch with more than 2^23 values of outputs."""
    T, E, D, F, n = 32, 8, 1536, 2048, ctypes.c_longlong()
    m = _lib.rm_fp4_moe(wt(mem, D), wt(mem, F), mem, mem, T, E, D, F)
    assert lib.rm_fp4_moe_workspace(m, B, ctypes.byref(n)) == OK
    assert n.value >= B * T * E * (D // 2 + D // 32 + F // 2 + F // 32 + 4 * D)
