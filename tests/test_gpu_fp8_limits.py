"""GPU tests of the 8-bit operators where their ranges end: GELU's far tail, sums of many samples, what is shared
between streams, and forms of the arguments that the products of ordinary layers do not take."""
from __future__ import annotations

import math

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300.api import (Fp8PFFN, Fp8Tensor, fp8_matmul, fp8_quantize, fp8_quantize_weight,
                                                     fp8_sync_status, fp8_wgrad)
from tests import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(y, want, tol, what):
    y, err = y.double(), (y.double() - want).abs()
    assert torch.isfinite(y).all(), f"{what}: {int((~torch.isfinite(y)).sum())} values are not finite"
    worst = (err / tol.clamp(min=1e-300)).max().item()
    print(f"{what}: worst error {worst:.3f} of its bound")
    assert worst <= 1, f"{what}: {int((err > tol).sum())} of {err.numel()} outside, worst {worst:.3g} of its bound"


def ok():
    assert fp8_sync_status() == _lib.RM_OK


# ---- GELU's far tail ------------------------------------------------------------------------------

# hidden values of whole blocks of 128
RANGES = [(-7, -6), (-9, -6), (-12.5, -10), (-5.5, -4.5), (-20, -13), (-1e4, -50), (-1e30, -1e28), (-6.5, 6.5), (-3, -2),
          (6, 50), (-3.4e38, -3e38), (-0.01, 0.01), (-8, -7)]


@pytest.mark.parametrize("B", [1, 20, 40, 100, 300])
def test_hidden_values_of_blocks_far_below_zero(B):
    """The input is zero, so the hidden pre-activations are the biases exactly.  Upper tail Q: GELU is off by |u| times
    3.5e-7 at most and times 1.6% of Q at most (1.5% of the fit, 2^-22 of the power of two, 8 steps in float32 of a
    logarithm below 2^7, each 2^-24 of it), and is zero where Q is no normal float (u below -12.85)."""
    T, D, F = 30, 16, 256                    # at 300 samples 180 tiles: more than are streamed
    lo, hi = (torch.tensor([RANGES[i % len(RANGES)][k] for i in range(2 * T)], dtype=torch.float64) for k in (0, 1))
    r = torch.rand((2 * T, 128), generator=gen(80), dtype=torch.float64)
    b1 = (lo[:, None] + (hi - lo)[:, None] * r).float().reshape(T, F).to(DEV)
    m = Fp8PFFN(torch.randn((T, D, F), generator=gen(81)).to(DEV), b1, torch.randn((T, F, D), generator=gen(82)).to(DEV),
                torch.zeros((T, D), device=DEV))
    X = torch.zeros((B, T, D), device=DEV)
    V, kept = m.forward_train(X, "f32")
    u = b1.double().expand(B, T, F)
    a, tail = ref.gelu(u), 0.5 * torch.special.erfc(u.abs() / math.sqrt(2.0))
    err = u.abs() * torch.minimum(torch.full_like(u, 3.5e-7), 0.016 * tail) + ref.UNIT_F32 * a.abs()
    err = torch.where(u < -12.85, a.abs(), err)
    scales = kept["a"].scales
    step = ref.pow2(scales[..., :2].to(torch.int64) - 127).repeat_interleave(128, -1)
    half = torch.maximum(ref.HALF["e4m3"] * (a.abs() + err), ref.LOWEST["e4m3"] / 2 * step)
    within(ref.value(kept["a"]), a, err + half, "kept a")
    top, off = (z.reshape(B, T, 2, 128).amax(-1) for z in (a.abs(), err))
    e = scales[..., :2].to(torch.int64) - 127
    low, high = ref.exponent((top - off).clamp(min=0), "e4m3"), ref.exponent(top + off, "e4m3")
    assert ((e >= low) & (e <= high) | (top <= off) & (e == 0)).all()
    assert torch.equal(m.forward(X, "f32"), V)
    ok()


# ---- long sums ----------------------------------------------------------------------------------------

def positive(shape, seed):
    """Values of one sign that share no grid."""
    return torch.exp(torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV))


@pytest.mark.parametrize("B", [1, 40])
def test_products_of_the_longest_sums(B):
    """Terms of one sign, K = 2^19: K / 32 instructions, each truncates what it adds and what it has, a unit in the last
    place (2^-23) of a running sum that is half the final one on average: K / 32 * 2^-23 = 2^-9."""
    K, N = 1 << 19, 16
    x, w = fp8_quantize(positive((B, 1, K), 83)), fp8_quantize_weight(positive((1, K, N), 84))
    want = ref.matmul(ref.value(x), ref.weight_value(w))
    within(fp8_matmul(x, w, None, "f32"), want, 2.0 ** -9 * want, "K = 2^19")
    ok()


def test_bf16_gradients_of_the_most_samples():
    """The same for B = 2^17 samples, 16 an instruction: B / 16 * 2^-23 = 2^-10, and half a step of bf16."""
    B, K, N = 1 << 17, 32, 24
    x, dy = fp8_quantize(positive((B, 1, K), 85)), positive((B, 1, N), 86).to(torch.bfloat16)
    dw, db = fp8_wgrad(x, dy, "bf16")
    want = ref.outer(ref.value(x), dy.double())
    within(dw, want, (2.0 ** -10 + ref.HALF_BF16) * want, "dW")
    assert abs(((dw.double() - want) / want).mean().item()) <= 2.0 ** -10
    want = dy.double().sum(0)
    within(db, want, (2.0 ** -10 + ref.HALF_BF16) * want, "db")
    ok()


def test_float32_gradients_of_millions_of_samples():
    """Float32 gradients are joined from sums of 2048 samples.  dW: within a chunk 128 instructions lose a unit in the
    last place each (2^-23) of a running sum of half the chunk's, 2^-17; 2049 chunks are added with rounding to nearest,
    half a unit (2^-24) of half the sum on average, 2^-14.  db, of one value that all samples share and that float32
    does not add exactly past 2^24 of its units: 256 additions in a chunk, which are exact, and the same 2049."""
    B, K, N = (1 << 22) + 65, 16, 8
    x = fp8_quantize(positive((B, 1, K), 87))
    dy = torch.full((B, 1, N), 129 / 128, dtype=torch.bfloat16, device=DEV)
    dw, db = fp8_wgrad(x, dy)
    want = ref.outer(ref.value(x), dy.double())
    within(db, dy.double().sum(0), 2.0 ** -14 * dy.double().sum(0), "db")
    within(dw, want, (2.0 ** -17 + 2.0 ** -14) * want, "dW")
    ok()
