"""Plain restatements of the 8-bit operators for the tests, in elementary torch operations:
the format bit by bit (float32 scaling by powers of two is exact, torch's cast rounds to nearest
even) and everything else in float64."""
from __future__ import annotations

import math

import torch

BLOCK = 128
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 9, "e5m2": 16}            # the largest value is 0.875 * 2^top
# half a step relative to the value, and the smallest step of a block with scale 1
HALF = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
LOWEST = {"e4m3": 2.0 ** -9, "e5m2": 2.0 ** -16}
HALF_BF16 = 2.0 ** -8
UNIT_F32 = 2.0 ** -24


def pow2(e: torch.Tensor) -> torch.Tensor:
    """2^e in float64, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def exponent(amax: torch.Tensor, fmt: str) -> torch.Tensor:
    """e of float64 maxima: the smallest whole number with amax <= largest * 2^e (0 for 0), at least -126."""
    largest = 0.875 * 2.0 ** TOP[fmt]
    m, x = torch.frexp(amax / largest)           # in [0.5, 1): amax / largest <= 2^x, and 2^(x-1) when m = 0.5
    e = torch.where(m == 0.5, x - 1, x).clamp(min=-126)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def quantise(x: torch.Tensor, fmt: str) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes as bytes [.., cols], E [.., blocks]) of CPU rows."""
    n = x.shape[-1]
    codes = torch.empty(x.shape, dtype=torch.uint8)
    es = []
    for j in range(0, n, BLOCK):
        v = x[..., j:j + BLOCK].double()
        fine = torch.isfinite(v)
        e = exponent(torch.where(fine, v.abs(), torch.zeros_like(v)).amax(-1), fmt)
        q = torch.where(fine, v / pow2(e).unsqueeze(-1), torch.full_like(v, math.nan)).float()
        codes[..., j:j + BLOCK] = q.to(F8[fmt]).view(torch.uint8)
        es.append(e + 127)
    return codes, torch.stack(es, -1).to(torch.uint8)


def quantise_weight(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes [T, K, N], E [T, kb, nb]) of a CPU weight."""
    T, K, N = w.shape
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    codes, E = torch.empty((T, K, N), dtype=torch.uint8), torch.empty((T, kb, nb), dtype=torch.uint8)
    for i in range(kb):
        for j in range(nb):
            v = w[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK].double()
            fine = torch.isfinite(v)
            e = exponent(torch.where(fine, v.abs(), torch.zeros_like(v)).amax((1, 2)), "e4m3")
            q = torch.where(fine, v / pow2(e)[:, None, None], torch.full_like(v, math.nan)).float()
            codes[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = q.to(F8["e4m3"]).view(torch.uint8)
            E[:, i, j] = (e + 127).to(torch.uint8)
    return codes, E


def value(q) -> torch.Tensor:
    """float64 values [.., cols] of 8-bit rows (an Fp8Tensor), on their device."""
    s = pow2(q.scales[..., :-(-q.cols // BLOCK)].to(torch.int64) - 127)
    return q.codes[..., :q.cols].double() * s.repeat_interleave(BLOCK, -1)[..., :q.cols]


def weight_value(q) -> torch.Tensor:
    """float64 values [T, K, N] of an 8-bit weight."""
    K, N = q.codes.shape[1], q.cols
    s = pow2(q.scales[..., :-(-N // BLOCK)].to(torch.int64) - 127)
    return q.codes[..., :N].double() * s.repeat_interleave(BLOCK, 1)[:, :K].repeat_interleave(BLOCK, 2)[..., :N]


def matmul(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """y[b, t, :] = x[b, t, :] w[t] in float64."""
    return torch.matmul(x.transpose(0, 1), w).transpose(0, 1)


def outer(x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    return torch.matmul(x.permute(1, 2, 0), y.transpose(0, 1))


def gelu(u: torch.Tensor) -> torch.Tensor:
    return 0.5 * u * torch.special.erfc(-u / math.sqrt(2.0))


def gelu_grad(u: torch.Tensor) -> torch.Tensor:
    return 0.5 * torch.special.erfc(-u / math.sqrt(2.0)) + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)


def sum_bound(n: int, absolute: torch.Tensor) -> torch.Tensor:
    """Bound on a float32 sum of n exact products of which the magnitudes add up to `absolute`: each of
    the n additions is off by at most one unit in the last place (2^-23, tensor cores truncate) of a
    partial sum that is at most `absolute`."""
    return (n + 1) * 2 * UNIT_F32 * absolute


def rounded(x: torch.Tensor, fmt: str = "e4m3") -> torch.Tensor:
    """float64 rows as their 8-bit form stands for them (CPU or GPU)."""
    n = x.shape[-1]
    out = torch.empty_like(x)
    for j in range(0, n, BLOCK):
        v = x[..., j:j + BLOCK]
        s = pow2(exponent(v.abs().amax(-1, keepdim=True), fmt))
        out[..., j:j + BLOCK] = (v / s).float().to(F8[fmt]).double() * s
    return out
