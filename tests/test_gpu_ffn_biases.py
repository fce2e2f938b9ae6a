"""GPU tests of the FFNs' biases as a program may hand them over."""
from __future__ import annotations

import pytest
import torch

from rankmixer_feature_interaction_gb300.api import Fp4MoE, Fp4PFFN, Fp8PFFN
from tests.test_gpu_experts import gates
from tests.test_gpu_fp4 import DEV, layer, ok, rows

pytestmark = pytest.mark.gpu


def shifted(b, by):
    """The same bias as a view that begins `by` elements into a buffer."""
    buf = torch.empty(b.numel() + by, dtype=b.dtype, device=DEV)
    buf[by:] = b.flatten()
    return buf[by:].view(b.shape)


@pytest.mark.parametrize("by", [1, 2, 4])
@pytest.mark.parametrize("kind", [Fp8PFFN, Fp4PFFN, Fp4MoE])
def test_biases_at_any_address(kind, by):
    T, E, D, F, B = 2, 3, 64, 96, 5
    w1, b1, w2, b2 = (v.to(DEV) for v in layer((T, E) if kind is Fp4MoE else (T,), D, F, 31))
    X = rows((B, T, D), 32).to(DEV)
    more = (gates(B, T, E, 0.5, 33).to(DEV),) if kind is Fp4MoE else ()
    moved = kind(w1, shifted(b1, by), w2, shifted(b2, by))
    assert torch.equal(moved.forward(X, *more), kind(w1, b1, w2, b2).forward(X, *more))
    ok()
