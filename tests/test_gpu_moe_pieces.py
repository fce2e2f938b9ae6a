"""GPU test of the Sparse-MoE FFN on 4-bit experts against its pieces, called one after another."""
from __future__ import annotations

import pytest
import torch

from rankmixer_feature_interaction_gb300.api import (Fp4MoE, expert_combine, expert_sort, fp4_expert_gather, fp4_expert_matmul,
                                                     fp4_quantize)
from tests import fp4_reference as ref
from tests.test_gpu_experts import HALF, gates
from tests.test_gpu_fp4 import DEV, layer, ok, rows, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,E,D,F", [(1, 1, 1, 32, 32), (8, 4, 8, 256, 160), (100, 3, 2, 96, 64), (129, 2, 4, 256, 96),
                                       (300, 2, 3, 512, 288), (900, 5, 4, 480, 96)])
def test_the_pieces_together_are_the_moe_ffn(B, T, E, D, F, out):
    """Rows sorted, gathered to 4 bits, layer 1, Gelu (torch, in float64), 4 bits, layer 2, combined: both that and the
    one call are the float64 sum over the open experts within float32 sums, what a hidden value next to a border may
    round to, a sum of E terms and one rounding to `out`.  The pieces keep the room of the open rows only."""
    w1, b1, w2, b2 = layer((T, E), D, F, 51)
    m = Fp4MoE(w1, b1, w2, b2)
    X, G = rows((B, T, D), 52, 0.5).to(torch.bfloat16).to(DEV), gates(B, T, E, 0.4, 53)
    G[0, 0] = 1.0                                    # some row is open
    G = G.to(DEV)
    r = expert_sort(G)
    n = r.count()
    u = fp4_expert_matmul(fp4_expert_gather(X, r, n), m.W1, r, m.b1, out_dtype="f32")
    a = fp4_quantize(ref.gelu(u.double()).float())
    pieces = expert_combine(fp4_expert_matmul(a, m.W2, r, m.b2, out_dtype="f32"), r, G, out_dtype=out)

    x, v1, v2, off = ref.value(fp4_quantize(X)), ref.weight_value(m.W1), ref.weight_value(m.W2), r.offsets.tolist()
    want, tol, total = (torch.zeros((B, T, D), dtype=torch.float64, device=DEV) for _ in range(3))
    for t in range(T):
        for e in range(E):
            b = torch.nonzero(G[:, t, e] > 0).flatten()
            assert off[t * E + e + 1] - off[t * E + e] == b.numel()
            if b.numel():
                y, d = ref.ffn(x[b, t], v1[t, e], b1[t, e].double(), v2[t, e], b2[t, e].double())
                g = G[b, t, e].double().unsqueeze(1)
                want[b, t] += g * y
                tol[b, t] += g * d
                total[b, t] += g * (y.abs() + d)
    tol += ref.sum_bound(E, total)
    assert want.abs().sum() > 0
    for what, V in (("pieces", pieces), ("one call", m.forward(X, G, out_dtype=out))):
        within(V, want, tol + (want.abs() + tol) * HALF[out], what)
    ok()
