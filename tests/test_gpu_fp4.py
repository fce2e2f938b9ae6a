"""GPU tests of the 4-bit operators against plain float64 restatements (tests/fp4_reference.py).

Rounding to 4 bits is checked bit for bit.  Products are checked element by element against the
float64 product of the same 4-bit values, within the bound of a float32 sum of that many terms and
half a step of the output's type; an FFN within what its hidden values may round to besides."""
from __future__ import annotations

import math

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300.api import (Fp4PFFN, Fp4Tensor, fp4_dequantize, fp4_matmul, fp4_quantize,
                                                     fp4_quantize_weight, fp8_sync_status)
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(shape, seed, spread=1.0):
    """Rows of differing size with a few large values."""
    g = gen(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g))
    return torch.where(torch.rand(shape, generator=g) < 0.01, 30 * x, x)


def weight(T, K, N, seed) -> Fp4Tensor:
    return fp4_quantize_weight((torch.randn((T, K, N), generator=gen(seed)) / math.sqrt(K)).to(DEV))


def within(y, want, tol, what):
    assert y.shape == want.shape, what
    if y.numel() == 0:
        return
    y, err = y.double(), (y.double() - want).abs()
    assert torch.isfinite(y).all(), f"{what}: {int((~torch.isfinite(y)).sum())} values are not finite"
    worst = (err / tol.clamp(min=1e-300)).max().item()
    print(f"{what}: worst error {worst:.3f} of its bound")
    assert worst <= 1, f"{what}: {int((err > tol).sum())} of {err.numel()} outside, worst {worst:.3g} of its bound"


def ok():
    assert fp8_sync_status() == _lib.RM_OK


# ---- to 4 bits and back -------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 3, 8), (2, 3, 31), (5, 2, 32), (3, 1, 33), (7, 5, 1003), (33, 4, 768),
                                   (1, 32, 1536), (257, 1, 400), (9, 300), (5,)])
def test_quantize_is_the_format_bit_for_bit(shape, dtype):
    x = rows(shape, 1, 3.0).to(DTYPES[dtype])
    q = fp4_quantize(x.to(DEV))
    code, E = ref.quantise(x)
    nb = E.shape[-1]
    assert q.shape == shape and torch.equal(q.scales[..., :nb].cpu(), E)
    assert torch.equal(q.codes.cpu(), ref.packed(code))
    for out in ("f32", "bf16"):
        y = fp4_dequantize(q, out)
        assert tuple(y.shape) == shape and torch.equal(y.double(), ref.value(q))
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_of_special_values(dtype):
    inf = float("inf")
    x = rows((16, 1, 70), 2)
    x[0] = 0
    x[1, 0, 5], x[1, 0, 40] = inf, -inf
    x[2, 0, :32] = float("nan")
    x[3, 0, 69] = float("nan")
    x[4, 0] = 2.0 ** -149
    x[5, 0] = 3.38e38
    x[6, 0] = 6.0
    x[7, 0] = 6.0 * (1 + 2.0 ** -7)
    x[8, 0] = torch.arange(70) * 2.0 ** -130
    x[9, 0] = (torch.arange(70) - 35) * 0.25                             # every tie
    x[10, 0] = -0.0
    x[11, 0] = 2.0 ** -126
    x[12, 0] = 1.5 * 2.0 ** 100
    x[13, 0] = 1.5 * (1 + 2.0 ** -7) * 2.0 ** 100
    x[14, 0, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) * torch.tensor([1, -1] * 16)
    x[15, 0] = 6.0 * 2.0 ** -127
    x = x.to(DTYPES[dtype])
    q = fp4_quantize(x.to(DEV))
    code, E = ref.quantise(x)
    assert torch.equal(q.scales[..., :3].cpu(), E)
    fine = (E != 255).unsqueeze(-1).expand(*E.shape, 16).flatten(-2)
    assert torch.equal(q.codes.cpu()[fine], ref.packed(code)[fine])
    y, nan = fp4_dequantize(q, "f32").cpu(), (E == 255).repeat_interleave(32, -1)[..., :70]
    assert torch.equal(y.isnan(), nan) and nan[1, 0, :64].all() and not nan[1, 0, 64:].any() and nan[3, 0, 64:].all()
    ok()


def test_restore_reads_any_exponent_byte():
    codes = torch.full((4, 1, 16), 0x23, dtype=torch.uint8).to(DEV)      # 1.5 and 1
    scales = torch.tensor([0, 1, 254, 255], dtype=torch.uint8).reshape(4, 1, 1).repeat(1, 1, 16).to(DEV)
    y = fp4_dequantize(Fp4Tensor(codes, scales, 32), "f32").cpu()[:, 0, :2].double()
    assert y[:3].tolist() == [[1.5 * 2.0 ** e, 2.0 ** e] for e in (-127, -126, 127)] and y[3].isnan().all()


def test_quantize_takes_strided_and_misaligned_rows_and_refuses_others():
    x = rows((6, 4, 300), 3).to(DEV)
    for v in (x[:, 1], x[..., 3:200], x[:, :, :128], x[::2, 0, 1:], x[2, 1], x[:, 2, 4:4 + 96].to(torch.bfloat16)):
        q, (code, E) = fp4_quantize(v), ref.quantise(v.cpu())
        assert torch.equal(q.codes.cpu(), ref.packed(code)) and torch.equal(q.scales.cpu()[..., :E.shape[-1]], E)
    with pytest.raises(ValueError):
        fp4_quantize(x.transpose(0, 2))
    with pytest.raises((ValueError, RuntimeError)):
        fp4_quantize(x[:, 1:3, :])                    # rows are not one stride apart
    with pytest.raises(ValueError):
        fp4_quantize(x.half())
    with pytest.raises(_lib.RankMixerError):
        fp4_quantize(x[:0])
    with pytest.raises(ValueError):
        fp4_dequantize(weight(1, 32, 32, 1))
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,gap", [(1, 0), (2, 1), (7, 0), (15, 2), (17, 0), (33, 0), (63, 5), (100, 1), (257, 0), (1003, 4)])
def test_rows_of_every_alignment(cols, gap, dtype):
    """Rows from each element of 16 bytes on, `gap` values apart: only they are read and only they are written."""
    n, ld, tdt, code = 37, cols + gap, DTYPES[dtype], {"bf16": _lib.RM_BF16, "f32": _lib.RM_F32}[dtype]
    for at in range(17 - 8 * (dtype == "f32")):
        size = at + (n - 1) * ld + cols
        flat = torch.full((size + 11,), float("nan"), dtype=tdt, device=DEV)
        v = flat[at:size].as_strided((n, cols), (ld, 1), at)
        x = rows((n, cols), 7 + at, 2.0).to(tdt)
        v.copy_(x)
        q, (c, E) = fp4_quantize(v), ref.quantise(x)
        assert torch.equal(q.codes.cpu(), ref.packed(c)) and torch.equal(q.scales.cpu()[..., :E.shape[-1]], E), at
        y = torch.full_like(flat, 5.0)
        _lib.rm_fp4_dequantize(q.c, n, cols, y[at:].data_ptr(), code, ld, torch.cuda.current_stream().cuda_stream)
        want = torch.full((size + 11,), 5.0, dtype=tdt)
        want.as_strided((n, cols), (ld, 1), at).copy_(ref.value(q).cpu())
        assert torch.equal(y.cpu(), want), at
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 128, 128), (3, 129, 127), (2, 200, 1001), (1, 400, 16), (5, 64, 256),
                                   (2, 3, 33, 40), (300, 20)])
def test_quantize_weight_is_the_format_bit_for_bit(shape, dtype):
    w = rows(shape, 4).to(DTYPES[dtype])
    q = fp4_quantize_weight(w.to(DEV))
    code, E = ref.quantise(w.transpose(-1, -2))
    nb = E.shape[-1]
    assert q.shape == shape and torch.equal(q.codes.cpu(), ref.packed(code))
    s = ref.weight_scales(q).cpu()
    assert torch.equal(s[..., :nb], E) and (s[..., nb:] == 127).all()
    assert torch.equal(ref.weight_value(q).cpu().float(),
                       ref.value(fp4_quantize(w.transpose(-1, -2).contiguous().to(DEV))).cpu().transpose(-1, -2).float())
    tail = q.scales.view(*q.scales.shape[:-1], 32, 4, 4).cpu()           # rows behind N: 127
    for r in range(shape[-1] % 128, 128 if shape[-1] % 128 else 0):
        assert (tail[..., -1, :, r % 32, r // 32, :] == 127).all()
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_weight_of_any_alignment(dtype):
    """Weights that begin one element off give the same as their copy."""
    buf = rows((2 * 96 * 130 + 1,), 30).to(DTYPES[dtype]).to(DEV)
    w = buf[1:].view(2, 96, 130)
    q, want = fp4_quantize_weight(w), fp4_quantize_weight(w.clone())
    assert w.data_ptr() % (2 * w.element_size()) and torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    ok()


def test_four_bits_past_32_bits():
    """More than 2^31 values, and rows behind the 2^31st."""
    n, C = 70001, 32000
    x = torch.zeros((n, C), dtype=torch.bfloat16, device=DEV)
    x[-1] = rows((C,), 5).to(torch.bfloat16).to(DEV)
    x[67109] = x[-1] * 3
    q = fp4_quantize(x)
    y = fp4_dequantize(q)
    for i in (-1, 67109, 0):
        assert torch.equal(y[i], fp4_dequantize(fp4_quantize(x[i])))
    code, E = ref.quantise(x[-1].cpu())
    assert torch.equal(q.codes[-1].cpu(), ref.packed(code)) and torch.equal(q.scales[-1, :C // 32].cpu(), E)
    assert int((y[1000:60000] != 0).sum()) == 0
    ok()


# ---- products -----------------------------------------------------------------------------------

SHAPES = [(1, 1, 1, 1), (1, 2, 32, 32), (3, 2, 33, 65), (8, 3, 256, 128), (5, 1, 512, 7), (16, 2, 300, 200), (17, 2, 64, 129),
          (64, 2, 1000, 96), (65, 1, 96, 300), (128, 3, 257, 256), (129, 2, 320, 264), (200, 3, 1003, 123), (256, 1, 768, 512),
          (300, 4, 512, 520), (1, 32, 1536, 640), (513, 2, 2080, 257), (1, 5, 6144, 130), (40, 7, 4097, 8), (700, 9, 96, 300)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,K,N", SHAPES)
def test_matmul(B, T, K, N, out):
    x, w = fp4_quantize(rows((B, T, K), 6, 0.5).to(DEV)), weight(T, K, N, 7)
    bias = torch.randn((T, N), generator=gen(8)).to(DEV) if (B + N) % 2 else None
    y = fp4_matmul(x, w, bias, out_dtype=out)
    xv, wv = ref.value(x), ref.weight_value(w)
    want, absolute = ref.matmul(xv, wv), ref.matmul(xv.abs(), wv.abs())
    if bias is not None:
        want, absolute = want + bias.double(), absolute + bias.double().abs()
    tol = ref.sum_bound(K + 1, absolute)
    within(y, want, tol + (want.abs() + tol) * ref.HALF_BF16 if out == "bf16" else tol + want.abs() * ref.UNIT_F32,
           f"matmul {B} {T} {K} {N} {out}")
    assert torch.equal(y, fp4_matmul(x, w, bias, out_dtype=out))         # the same bits again
    ok()


@pytest.mark.parametrize("B,T,K,N", [(7, 2, 320, 160), (300, 2, 320, 160)])
def test_matmul_scales_of_any_size_and_nan_blocks(B, T, K, N):
    """Exponents far apart, a block that is NaN in one row, and one in a weight's column: they stay there."""
    x = rows((B, T, K), 9, 0.5) * torch.exp2(torch.randint(-40, 40, (B, T, 1), generator=gen(10)).float())
    x[2, 1, 40] = float("inf")
    w = torch.randn((T, K, N), generator=gen(11)) * torch.exp2(torch.randint(-30, 30, (T, 1, N), generator=gen(12)).float())
    w[0, 300, 5] = float("nan")
    x4, w4 = fp4_quantize(x.to(DEV)), fp4_quantize_weight(w.to(DEV))
    y = fp4_matmul(x4, w4, out_dtype="f32")
    nan = torch.zeros((B, T, N), dtype=torch.bool, device=DEV)
    nan[2, 1] = True
    nan[:, 0, 5] = True
    assert torch.equal(y.isnan(), nan)
    x[2, 1, 40], w[0, 300, 5] = 1.0, 1.0
    xv, wv = ref.value(fp4_quantize(x.to(DEV))), ref.weight_value(fp4_quantize_weight(w.to(DEV)))
    want, tol = ref.matmul(xv, wv), ref.sum_bound(K + 1, ref.matmul(xv.abs(), wv.abs()))
    within(torch.where(nan, want, y.double()), want, tol + want.abs() * ref.UNIT_F32, "scales")
    ok()


@pytest.mark.parametrize("B", [4, 300])
def test_padding_is_not_read(B):
    """Bytes behind a row's blocks (codes and scales) hold anything, NaN scales among it."""
    T, K, N = 2, 96, 40
    x, w = rows((B, T, K), 13).to(DEV), weight(T, K, N, 14)
    q = fp4_quantize(x)
    codes = torch.full((B, T, 80), 0xff, dtype=torch.uint8, device=DEV)
    scales = torch.full((B, T, 32), 0xff, dtype=torch.uint8, device=DEV)
    codes[..., :48], scales[..., :3] = q.codes[..., :48], q.scales[..., :3]
    assert torch.equal(fp4_matmul(Fp4Tensor(codes, scales, K), w), fp4_matmul(q, w))
    assert torch.equal(fp4_dequantize(Fp4Tensor(codes, scales, K)), fp4_dequantize(q))
    ok()


@pytest.mark.parametrize("B,N", [(3, 40), (130, 41), (257, 264)])
def test_matmul_writes_only_its_output(B, N):
    """Rows around Y keep what they held."""
    T, K = 2, 64
    x, w = fp4_quantize(rows((B, T, K), 15).to(DEV)), weight(T, K, N, 16)
    buf = torch.full((B * T * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = buf[32:32 + B * T * N]
    _lib.rm_fp4_matmul(x.c, w.c, None, y.data_ptr(), _lib.RM_BF16, B, T, K, N, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(y.view(B, T, N), fp4_matmul(x, w)) and (buf[:32] == 7).all() and (buf[32 + B * T * N:] == 7).all()
    ok()


# ---- FFN ----------------------------------------------------------------------------------------

def layer(lead, D, F, seed):
    g = gen(seed)
    w1 = torch.randn((*lead, D, F), generator=g) / math.sqrt(D)
    w2 = torch.randn((*lead, F, D), generator=g) / math.sqrt(F)
    b1, b2 = 0.1 * torch.randn((*lead, F), generator=g), 0.1 * torch.randn((*lead, D), generator=g)
    return [v.to(DEV) for v in (w1, b1, w2, b2)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,F", [(1, 1, 32, 32), (3, 2, 64, 160), (16, 2, 256, 512), (33, 1, 96, 288), (100, 2, 128, 256),
                                     (130, 3, 320, 1056), (300, 2, 512, 512), (1, 8, 768, 1536),
                                     # many rows by pairs of CTAs, hidden layers that fill part of a tile
                                     (5000, 4, 64, 32), (2600, 8, 32, 96), (2600, 4, 96, 160), (2600, 4, 224, 288)])
def test_pffn(B, T, D, F, x_dtype, out):
    w1, b1, w2, b2 = layer((T,), D, F, 20)
    f = Fp4PFFN(w1, b1, w2, b2)
    X = rows((B, T, D), 21, 0.5).to(DTYPES[x_dtype]).to(DEV)
    V = f.forward(X, out_dtype=out)
    x, v1, v2 = ref.value(fp4_quantize(X)), ref.weight_value(f.W1), ref.weight_value(f.W2)
    for t in range(T):
        want, tol = ref.ffn(x[:, t], v1[t], b1[t].double(), v2[t], b2[t].double())
        half = ref.HALF_BF16 if out == "bf16" else ref.UNIT_F32
        within(V[:, t], want, tol + (want.abs() + tol) * half, f"pffn token {t}")
    assert torch.equal(V, f.forward(X, out_dtype=out))
    ok()


def test_pffn_where_gelu_is_far_below_zero():
    """Hidden blocks all far in Gelu's tail still have scales of their own."""
    T, D, F, B = 1, 64, 64, 40
    w1, b1, w2, b2 = layer((T,), D, F, 22)
    b1 = b1 * 0 - torch.linspace(0, 12, F, device=DEV)
    f = Fp4PFFN(w1 * 0.01, b1, w2, b2 * 0)
    X = rows((B, T, D), 23, 0.1).to(DEV)
    V = f.forward(X, out_dtype="f32")
    want, tol = ref.ffn(ref.value(fp4_quantize(X))[:, 0], ref.weight_value(f.W1)[0], b1[0].double(),
                        ref.weight_value(f.W2)[0], b2[0].double() * 0)
    within(V[:, 0], want, tol + want.abs() * ref.UNIT_F32, "tail")
    ok()
