"""GPU tests of what the Sparse-MoE FFN on 4-bit experts holds in float32."""
from __future__ import annotations

import pytest
import torch

from rankmixer_feature_interaction_gb300.api import Fp4MoE
from tests import fp4_reference as ref
from tests.test_gpu_experts import HALF, gates
from tests.test_gpu_fp4 import DEV, gen, ok, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_experts_outputs_keep_float32_whatever_the_batch(out):
    """Experts whose outputs are known: W1 is zero and b1 holds 4-bit numbers from 8 on, of which Gelu is the number
    itself in float32, so the hidden values are b1; 32 products of numbers of four bits under one scale a column add
    up exactly, and the bias is rounded in once (2^-24).  Left is a float32 sum of E terms, one rounding to `out`, and
    no difference between a sample served alone, with few and with many (400: more than 2^23 values of outputs)."""
    T, E, D, F, B = 4, 8, 1024, 32, 400
    g = gen(90)
    b1 = 4.0 * torch.randint(2, 5, (T, E, F), generator=g).float()
    w2, b2 = torch.randn((T, E, F, D), generator=g), torch.randn((T, E, D), generator=g)
    m = Fp4MoE(torch.zeros((T, E, D, F), device=DEV), b1.to(DEV), w2.to(DEV), b2.to(DEV))
    X, G = torch.randn((B, T, D), generator=g).to(DEV), gates(B, T, E, 0.4, 91).to(DEV)
    assert B * T * E * D > 1 << 23 > 10 * T * E * D
    y = torch.einsum("tef,tefd->ted", b1.double().to(DEV), ref.weight_value(m.W2)) + b2.double().to(DEV)
    V = m.forward(X, G, out_dtype=out)
    want, size = torch.einsum("bte,ted->btd", G.double(), y), torch.einsum("bte,ted->btd", G.double(), y.abs())
    # an expert's output is within 2^-24 of itself, which is half of what one more term is allowed
    tol = ref.sum_bound(E + 1, size)
    within(V, want, tol + (want.abs() + tol) * HALF[out], "V")
    for part in (slice(0, 1), slice(3, 13), slice(100, 350)):
        assert torch.equal(m.forward(X[part].contiguous(), G[part].contiguous(), out_dtype=out), V[part])
    ok()
