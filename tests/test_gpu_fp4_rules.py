"""GPU tests of 4-bit FFNs around the sizes at which one kernel takes over from another."""
from __future__ import annotations

import pytest
import torch

from rankmixer_feature_interaction_gb300.api import Fp4PFFN, fp4_quantize
from tests import fp4_reference as ref
from tests.test_gpu_experts import HALF
from tests.test_gpu_fp4 import DEV, layer, ok, rows, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [64, 79, 80, 81, 97, 113, 127, 128, 129])
@pytest.mark.parametrize("T,D,F", [(20, 64, 1024), (3, 96, 320)])
def test_ffns_of_about_a_tile_of_rows(B, T, D, F):
    """More and fewer tiles than SMs: streamed, and by pairs of CTAs."""
    w1, b1, w2, b2 = layer((T,), D, F, 41)
    f = Fp4PFFN(w1, b1, w2, b2)
    X = rows((B, T, D), 42, 0.5).to(DEV)
    x, v1, v2 = ref.value(fp4_quantize(X)), ref.weight_value(f.W1), ref.weight_value(f.W2)
    for out in ("f32", "bf16"):
        V = f.forward(X, out)
        for t in range(T):
            want, tol = ref.ffn(x[:, t], v1[t], b1[t].double(), v2[t], b2[t].double())
            within(V[:, t], want, tol + (want.abs() + tol) * HALF[out], f"token {t} {out}")
    ok()
