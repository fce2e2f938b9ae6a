"""GPU tests of 4-bit products whose rows of outputs are longer than 2^31 bytes."""
from __future__ import annotations

import pytest
import torch

from rankmixer_feature_interaction_gb300.api import expert_sort, fp4_expert_gather, fp4_expert_matmul, fp4_quantize_weight
from tests.test_gpu_fp4 import DEV, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out,N", [("f32", (1 << 29) + 296), ("bf16", (1 << 30) + 296), ("f32", (1 << 29) - 24)])
def test_experts_products_of_rows_past_2_to_31_bytes(out, N):
    """33 sorted rows, of which 32 fill a warp's piece of a tile: a column's bytes pass what a TMA coordinate holds (in
    the last case they just do not).  K = 1 and 4-bit numbers, so every output is one exact product."""
    B, n = 200, 33
    G = torch.zeros((B, 1, 1), device=DEV)
    G[7:7 + n] = 1
    r = expert_sort(G)
    numbers = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    X = numbers[torch.arange(B, device=DEV) % 7].view(B, 1, 1)
    W = numbers.to(torch.bfloat16).repeat(N // 7 + 1)[:N].view(1, 1, 1, N)
    w = fp4_quantize_weight(W)
    x = fp4_expert_gather(X, r, n)
    y = fp4_expert_matmul(x, w, r, out_dtype=out)
    assert y.shape == (n, N)
    edge = (1 << 31) // y.element_size()
    for at in (0, 1 << 20, N // 2, min(edge, N) - 4096, edge - 256, N - 4096):
        part = slice(at, min(at + 4096, N))
        want = X[7:7 + n, 0] * W[0, 0, :, part].float()
        assert torch.equal(y[:, part].float(), want), at
    del y
    ok()
