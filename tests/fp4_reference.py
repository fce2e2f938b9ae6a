"""Plain restatements of the 4-bit operators and of the experts' rows for the tests: the format value
by value from its definition, sorting by Python's loops over what torch.nonzero gives, everything else
in float64."""
from __future__ import annotations

import math

import torch

BLOCK = 32
NUMBERS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
HALF_BF16 = 2.0 ** -8
UNIT_F32 = 2.0 ** -24


def pow2(e: torch.Tensor) -> torch.Tensor:
    """2^e in float64, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def blocks(x: torch.Tensor) -> torch.Tensor:
    n = x.shape[-1]
    return torch.nn.functional.pad(x.double(), [0, -n % BLOCK]).unflatten(-1, (-1, BLOCK))


def exponent(amax: torch.Tensor) -> torch.Tensor:
    """e of finite float64 maxima: the smallest whole number with amax <= 6 * 2^e (0 for 0), at least -126."""
    m, x = torch.frexp(amax / 6)                 # amax / 6 <= 2^x, and 2^(x - 1) when m = 0.5
    # the quotient is rounded: a maximum just above 6 * 2^e must not pass for 6 * 2^e itself
    e = torch.where((m == 0.5) & (amax <= 6 * pow2(x.clamp(-1000, 1000) - 1)), x - 1, x).clamp(min=-126)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def nearest(a: torch.Tensor) -> torch.Tensor:
    """Index of the nearest of NUMBERS to magnitudes in [0, 6], ties to the even index."""
    numbers = NUMBERS.to(a.device)
    hi = torch.bucketize(a, numbers).clamp(1, 7)              # numbers[hi - 1] < a <= numbers[hi]
    lo = hi - 1
    down, up = a - numbers[lo], numbers[hi] - a
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes [.., blocks, 32], E [.., blocks]) of rows; a block that is not finite has E = 255 and any codes."""
    v = blocks(x)
    fine = torch.isfinite(v).all(-1)
    e = exponent(torch.where(fine, v.abs().amax(-1), torch.zeros_like(v[..., 0])))
    q = torch.where(fine.unsqueeze(-1), v / pow2(e).unsqueeze(-1), torch.zeros_like(v))
    code = nearest(q.abs()) + 8 * torch.signbit(q).long()
    return code.to(torch.uint8), torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)


def packed(code: torch.Tensor) -> torch.Tensor:
    """Bytes [.., 16 blocks] of codes [.., blocks, 32]."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).flatten(-2)


def _numbers(bytes_: torch.Tensor) -> torch.Tensor:
    code = torch.stack([bytes_ & 15, bytes_ >> 4], -1).flatten(-2).long()
    return NUMBERS.to(code.device)[code % 8] * torch.where(code >= 8, -1.0, 1.0).double()


def value(q) -> torch.Tensor:
    """float64 values [.., cols] of 4-bit rows (an Fp4Tensor of activations), on their device."""
    nb = -(-q.cols // BLOCK)
    E = q.scales[..., :nb].to(torch.int64)
    s = torch.where(E == 255, torch.full_like(E, 0).double() * math.nan, pow2(E - 127))
    return (_numbers(q.codes[..., :16 * nb]).unflatten(-1, (nb, BLOCK)) * s.unsqueeze(-1)).flatten(-2)[..., :q.cols]


def weight_scales(q) -> torch.Tensor:
    """E [.., N, blocks of K] of a 4-bit weight, out of the tensor cores' order (with the padding of the last 256)."""
    s = q.scales.view(*q.scales.shape[:-1], 32, 4, 4)         # [.., tile, quad, r % 32, r / 32, block]
    s = s.movedim(-2, -3).flatten(-3, -2)                     # [.., tile, quad, r, block]
    return s.movedim(-2, -3).flatten(-4, -3).flatten(-2)[..., :q.cs[-2], :]


def weight_value(q) -> torch.Tensor:
    """float64 values [.., K, N] of a 4-bit weight."""
    nb = -(-q.cols // BLOCK)
    s = pow2(weight_scales(q)[..., :nb].to(torch.int64) - 127)
    v = (_numbers(q.codes[..., :16 * nb]).unflatten(-1, (nb, BLOCK)) * s.unsqueeze(-1)).flatten(-2)[..., :q.cols]
    return v.transpose(-1, -2)


def matmul(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """y[b, t, :] = x[b, t, :] w[t] in float64."""
    return torch.matmul(x.transpose(0, 1), w).transpose(0, 1)


def gelu(u: torch.Tensor) -> torch.Tensor:
    return 0.5 * u * torch.special.erfc(-u / math.sqrt(2.0))


def sum_bound(n: int, absolute: torch.Tensor) -> torch.Tensor:
    """Bound on a float32 sum of n exact products of which the magnitudes add up to `absolute`: each of
    the n additions is off by at most one unit in the last place (2^-23, tensor cores truncate) of a
    partial sum that is at most `absolute`."""
    return (n + 1) * 2 * UNIT_F32 * absolute


def rounded_between(g: torch.Tensor, err: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Q(g), lowest, highest) of float64 rows known to within err: every value of a block within its
    error, the block's exponent as small and as large as that allows.  Rounding is monotone, so what a
    kernel gives for values within err lies between."""
    n = g.shape[-1]
    v, d = blocks(g), blocks(err)
    top = v.abs()

    def q(x, e):
        s = pow2(e).unsqueeze(-1)
        y = (x / s).clamp(-6, 6)
        return torch.copysign(NUMBERS.to(x.device)[nearest(y.abs())], y) * s

    e = exponent(top.amax(-1))
    small, large = exponent((top - d).clamp(min=0).amax(-1)), exponent((top + d).amax(-1))
    # an exponent of 0 stands for a block that may be all zeros: its values are then at most err
    lo = torch.minimum(q(v - d, small), q(v - d, large))
    hi = torch.maximum(q(v + d, small), q(v + d, large))
    return tuple(x.flatten(-2)[..., :n] for x in (q(v, e), lo, hi))


def ffn(x: torch.Tensor, w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, b2: torch.Tensor):
    """(v, bound) of one FFN on 4-bit values: x [rows, D] (already rounded), w1 [D, F], w2 [F, D], all
    float64.  bound: of float32 sums, of Gelu within 3.5e-7 |u| + 2^-24, and of what a hidden value
    near a border may round to."""
    u = x @ w1 + b1
    # bias added in float32, and |Gelu'| <= 1.13
    du = sum_bound(w1.shape[0] + 1, x.abs() @ w1.abs() + b1.abs())
    a, lo, hi = rounded_between(gelu(u), 1.13 * du + 4e-7 * u.abs() + 1e-30)
    v = a @ w2 + b2
    most = torch.maximum(lo.abs(), hi.abs())
    return v, (torch.maximum(hi - a, a - lo)) @ w2.abs() + sum_bound(w2.shape[0] + 1, most @ w2.abs() + b2.abs())


def sorted_rows(G: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(offsets, source, slot) of gates [B, T, E] on the CPU, one open gate after another."""
    B, T, E = G.shape
    slot = torch.full((B, T, E), -1, dtype=torch.int32)
    offsets, source = [0], []
    for t in range(T):
        for e in range(E):
            for b in torch.nonzero(G[:, t, e] > 0).flatten().tolist():
                slot[b, t, e] = len(source)
                source.append(b * T + t)
            offsets.append(len(source))
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(source, dtype=torch.int32), slot
