"""GPU tests of the 8-bit operators against plain float64 restatements (tests/fp8_reference.py).

Saving in 8 bits is checked bit for bit.  Products are checked element by element against the
float64 product of the same 8-bit values, within the bound of a float32 sum of that many terms and
half a step of the output's type.  The FFN's stages are checked one by one from what it keeps, so
that a value at the border between two codes cannot hide or fake an error."""
from __future__ import annotations

import math

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib, api
from rankmixer_feature_interaction_gb300.api import (Fp8PFFN, Fp8Tensor, fp8_dequantize, fp8_matmul, fp8_quantize,
                                                     fp8_quantize_weight, fp8_sync_status, fp8_wgrad)
from tests import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(shape, seed, spread=3.0):
    """Rows of differing size with a few large values."""
    g = gen(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g))
    return torch.where(torch.rand(shape, generator=g) < 0.01, 30 * x, x)


def act(shape, seed, fmt="e4m3", spread=0.5) -> Fp8Tensor:
    return fp8_quantize(rows(shape, seed, spread).to(DEV), fmt)


def weight(T, K, N, seed) -> Fp8Tensor:
    return fp8_quantize_weight((torch.randn((T, K, N), generator=gen(seed)) / math.sqrt(K)).to(DEV))


def within(y, want, tol, what):
    y, err = y.double(), (y.double() - want).abs()
    assert torch.isfinite(y).all(), f"{what}: {int((~torch.isfinite(y)).sum())} values are not finite"
    worst = (err / tol.clamp(min=1e-300)).max().item()
    print(f"{what}: worst error {worst:.3f} of its bound")
    assert worst <= 1, f"{what}: {int((err > tol).sum())} of {err.numel()} outside, worst {worst:.3g} of its bound"


def ok():
    assert fp8_sync_status() == _lib.RM_OK


# ---- save and restore ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 3, 8), (2, 3, 127), (5, 2, 128), (3, 1, 129), (7, 5, 1003), (33, 4, 768),
                                   (1, 32, 1536), (257, 1, 400)])
def test_quantize_is_the_format_bit_for_bit(shape, dtype, fmt):
    x = rows(shape, 1).to(DTYPES[dtype])
    q = fp8_quantize(x.to(DEV), fmt)
    codes, E = ref.quantise(x, fmt)
    n, nb = shape[-1], E.shape[-1]
    assert torch.equal(q.scales[..., :nb].cpu(), E)
    assert torch.equal(q.codes.view(torch.uint8)[..., :n].cpu(), codes)
    for out in ("f32", "bf16"):
        y = fp8_dequantize(q, out)
        assert tuple(y.shape) == shape and torch.equal(y.double(), ref.value(q))
    ok()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_of_special_values(fmt):
    big, inf = 0.875 * 2.0 ** ref.TOP[fmt], float("inf")
    x = rows((14, 1, 260), 2, 1.0)
    x[0] = 0
    x[1, 0, 5], x[1, 0, 200] = inf, -inf
    x[2, 0, :128] = float("nan")
    x[3, 0] = inf
    x[4, 0] = 2.0 ** -149
    x[5, 0] = 3.4e38
    x[6, 0, :130] = big
    x[7, 0, :130] = big * (1 + 2.0 ** -22)
    x[8, 0] = torch.arange(260) * 2.0 ** -140
    x[9, 0] = (torch.arange(260) - 130) * (big / 4096) * 0.5           # ties and subnormal codes
    x[10, 0, ::2] = -0.0
    x[11, 0] = 2.0 ** -126
    x[12, 0] = 1.75 * 2.0 ** 100
    x[13, 0] = 1.7500001 * 2.0 ** 100
    q = fp8_quantize(x.to(DEV), fmt)
    codes, E = ref.quantise(x, fmt)
    assert torch.equal(q.scales[..., :3].cpu(), E)
    got = q.codes.view(torch.uint8)[..., :260].cpu()
    nan = codes.view(ref.F8[fmt]).double().isnan()
    assert torch.equal(got.view(ref.F8[fmt]).double().isnan(), nan)      # any NaN code will do
    assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, codes))
    y = fp8_dequantize(q, "f32").cpu()
    assert torch.equal(y.isnan(), nan)
    ok()


def test_restore_reads_any_exponent_byte():
    codes = torch.full((4, 1, 16), 1.5).to(torch.float8_e4m3fn).to(DEV)
    scales = torch.tensor([0, 1, 254, 255], dtype=torch.uint8).reshape(4, 1, 1).repeat(1, 1, 4).to(DEV)
    y = fp8_dequantize(Fp8Tensor(codes, scales, 16), "f32").cpu()[:, 0, 0].double()
    assert y[0] == 1.5 * 2.0 ** -127 and y[1] == 1.5 * 2.0 ** -126 and y[2] == 1.5 * 2.0 ** 127 and y[3].isnan()


def test_quantize_takes_strided_and_misaligned_rows_and_refuses_others():
    x = rows((6, 4, 300), 3).to(DEV)
    for v in (x[:, 1], x[..., 3:200], x[:, :, :128], x[::2, 0, 1:], x[2, 1]):
        q, (codes, E) = fp8_quantize(v), ref.quantise(v.cpu().reshape(-1, v.shape[-1]), "e4m3")
        assert torch.equal(q.codes.view(torch.uint8)[..., :v.shape[-1]].cpu().reshape(codes.shape), codes)
        assert torch.equal(q.scales.cpu()[..., :E.shape[-1]].reshape(E.shape), E)
    with pytest.raises(ValueError):
        fp8_quantize(x.transpose(0, 2))
    with pytest.raises((ValueError, RuntimeError)):
        fp8_quantize(x[:, 1:3, :])                    # rows are not one stride apart
    with pytest.raises(ValueError):
        fp8_quantize(x.half())
    with pytest.raises(_lib.RankMixerError):
        fp8_quantize(x[:0])
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(1, 1, 1), (2, 128, 128), (3, 129, 127), (2, 200, 1001), (1, 400, 16), (5, 64, 256)])
def test_quantize_weight_is_the_format_bit_for_bit(T, K, N, dtype):
    w = rows((T, K, N), 4, 1.0).to(DTYPES[dtype])
    w[0, 0, 0] = 0 if K * N == 1 else float("inf")
    q = fp8_quantize_weight(w.to(DEV))
    codes, E = ref.quantise_weight(w)
    assert torch.equal(q.scales[..., :E.shape[-1]].cpu(), E)
    assert torch.equal(q.codes.view(torch.uint8)[..., :N].cpu(), codes)
    ok()


def test_save_and_restore_past_32_bits():
    """More than 2^32 values in one call: the last rows land where they belong."""
    n, C = (1 << 23) + 5, 520                           # 4.36e9 values, 8.7 GB in bf16
    x = torch.zeros((n, C), dtype=torch.bfloat16, device=DEV)
    tail = rows((7, C), 5).to(torch.bfloat16)
    x[-7:] = tail.to(DEV)
    q = fp8_quantize(x)
    codes, E = ref.quantise(tail, "e4m3")
    assert torch.equal(q.codes.view(torch.uint8)[-7:, :C].cpu(), codes) and torch.equal(q.scales[-7:, :5].cpu(), E)
    del x
    y = fp8_dequantize(q)
    assert torch.equal(y[-7:].double(), ref.value(Fp8Tensor(q.codes[-7:], q.scales[-7:], C)))
    assert not y[:1000].any()
    ok()


# ---- products -------------------------------------------------------------------------------------

SIZES = [(1, 1, 1, 1), (1, 3, 16, 8), (2, 2, 128, 128), (1, 32, 256, 512), (5, 3, 200, 72), (16, 2, 384, 256),
         (17, 1, 130, 257), (33, 2, 1000, 713), (64, 4, 512, 640), (100, 2, 257, 129), (128, 3, 128, 384), (129, 2, 640, 256),
         (200, 1, 1536, 300), (256, 2, 256, 256), (333, 3, 272, 1001), (513, 2, 128, 520), (1000, 1, 96, 128)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("B,T,K,N", SIZES)
def test_matmul(B, T, K, N, trans, out):
    fmt = "e5m2" if trans else "e4m3"
    x = act((B, T, K), 6, fmt)
    w = weight(T, N, K, 7) if trans else weight(T, K, N, 7)
    bias = torch.randn((T, N), generator=gen(8)).to(DEV) if (B + N) % 2 else None
    y = fp8_matmul(x, w, bias, out, trans)
    xv, wv = ref.value(x), ref.weight_value(w)
    wv = wv.transpose(1, 2) if trans else wv
    want, size = ref.matmul(xv, wv), ref.matmul(xv.abs(), wv.abs())
    tol = ref.sum_bound(K, size)
    if bias is not None:
        want = want + bias.double()
        tol = tol + 2 * ref.UNIT_F32 * (size + bias.double().abs())
    if out == "bf16":
        tol = tol + ref.HALF_BF16 * (want.abs() + tol)
    assert tuple(y.shape) == (B, T, N) and y.dtype == DTYPES[out]
    within(y, want, tol, f"matmul {B} {T} {K} {N} trans={trans} {out}")
    ok()


def test_matmul_applies_every_exponent():
    """Codes of one, exponents that differ from block to block and row to row: sums of powers of two, exact."""
    for B in (3, 200):
        T, K, N = 2, 520, 400
        g = gen(9)
        one = torch.ones(1).to(torch.float8_e4m3fn).view(torch.uint8).item()
        E = torch.randint(125, 130, (B, T, 8), generator=g, dtype=torch.uint8)
        Ew = torch.randint(125, 130, (T, 5, 4), generator=g, dtype=torch.uint8)
        x = Fp8Tensor(torch.full((B, T, 528), one, dtype=torch.uint8).view(torch.float8_e4m3fn).to(DEV), E.to(DEV), K)
        w = Fp8Tensor(torch.full((T, K, N), one, dtype=torch.uint8).view(torch.float8_e4m3fn).to(DEV), Ew.to(DEV), N)
        assert torch.equal(fp8_matmul(x, w, None, "f32").double(), ref.matmul(ref.value(x), ref.weight_value(w)))
        Ewt = torch.randint(125, 130, (T, 4, 8), generator=g, dtype=torch.uint8)
        w = Fp8Tensor(torch.full((T, N, 528), one, dtype=torch.uint8).view(torch.float8_e4m3fn).to(DEV), Ewt.to(DEV), K)
        assert torch.equal(fp8_matmul(x, w, None, "f32", True).double(),
                           ref.matmul(ref.value(x), ref.weight_value(w).transpose(1, 2)))
    ok()


@pytest.mark.parametrize("B", [3, 40, 300])
def test_matmul_keeps_nan_in_its_row_and_reads_no_padding(B):
    T, K, N = 2, 200, 136
    xs = rows((B, T, K), 10, 0.5)
    xs[1, 1, 17] = float("nan")
    x, w = fp8_quantize(xs.to(DEV)), weight(T, K, N, 11)
    x.codes.view(torch.uint8)[..., K:] = 0x7f           # NaN codes in the padding of both operands
    x.scales[..., 2:] = 255
    wide = torch.full((T, K, 144), 0x7f, dtype=torch.uint8, device=DEV)
    wide[..., :N] = w.codes.view(torch.uint8)[..., :N]
    w = Fp8Tensor(wide.view(torch.float8_e4m3fn), torch.where(torch.arange(4, device=DEV) < 2, w.scales, 255).to(torch.uint8), N)
    y = fp8_matmul(x, w, None, "f32")
    bad = torch.zeros((B, T, 1), dtype=torch.bool, device=DEV)
    bad[1, 1] = True
    assert torch.equal(y.isnan(), bad.expand(B, T, N))
    ok()


def test_matmul_with_codes_past_32_bits():
    B, T, K, N = 8193, 8, 65600, 16                       # 4.3e9 codes
    x = Fp8Tensor(torch.zeros((B, T, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                  torch.full((B, T, 516), 127, dtype=torch.uint8, device=DEV), K)
    tail = act((3, T, K), 12)
    x.codes.view(torch.uint8)[-3:] = tail.codes.view(torch.uint8)
    x.scales[-3:] = tail.scales
    w = weight(T, K, N, 13)
    y = fp8_matmul(x, w, None, "f32")
    assert not y[:-3].any()
    xv, wv = ref.value(tail), ref.weight_value(w)
    within(y[-3:], ref.matmul(xv, wv), ref.sum_bound(K, ref.matmul(xv.abs(), wv.abs())), "past 32 bits")
    ok()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,K,N", [(1, 1, 1, 8), (1, 3, 16, 16), (5, 2, 128, 128), (64, 2, 256, 256), (65, 1, 130, 264),
                                     (130, 3, 272, 520), (777, 2, 528, 1040), (1000, 1, 1001, 40), (2048, 1, 256, 512)])
def test_wgrad(B, T, K, N, out):
    x, dy = act((B, T, K), 14), (rows((B, T, N), 15, 0.5) / B).to(torch.bfloat16).to(DEV)
    dw, db = fp8_wgrad(x, dy, out)
    xv, yv = ref.value(x), dy.double()
    for got, want, size, what in ((dw, ref.outer(xv, yv), ref.outer(xv.abs(), yv.abs()), "dW"),
                                  (db, yv.sum(0), yv.abs().sum(0), "db")):
        tol = ref.sum_bound(B, size)
        if out == "bf16":
            tol = tol + ref.HALF_BF16 * (want.abs() + tol)
        assert got.dtype == DTYPES[out] and got.shape == want.shape
        within(got, want, tol, f"{what} {B} {T} {K} {N} {out}")
    ok()


def test_wgrad_padding_and_nan_stay_where_they_are():
    B, T, K, N = 70, 2, 200, 136
    x, dy = act((B, T, K), 16), rows((B, T, N), 17, 0.5).to(torch.bfloat16).to(DEV)
    x.codes.view(torch.uint8)[..., K:] = 0x7f
    x.scales[..., 2:] = 255
    dy[3, 1, 5] = float("nan")
    x.codes.view(torch.uint8)[9, 0, 150] = 0x7f
    dw, db = fp8_wgrad(x, dy)
    bad = torch.zeros((T, K, N), dtype=torch.bool, device=DEV)
    bad[1, :, 5] = True
    bad[0, 150, :] = True
    assert torch.equal(dw.isnan(), bad)
    assert db.isnan().sum() == 1 and db[1, 5].isnan()
    ok()


def test_wgrad_restores_codes_of_any_size():
    """Exponents from tiny to huge: the restored operand is exact, so one-sample gradients are products exact in float32."""
    T, K, N = 1, 256, 16
    codes = torch.arange(256, dtype=torch.uint8).repeat(120, 1, 1)
    codes[..., 0x7f] = codes[..., 0xff] = 0
    E = torch.arange(68, 188, dtype=torch.uint8).reshape(120, 1, 1).repeat(1, 1, 4)
    for b in (0, 59, 60, 119):
        x = Fp8Tensor(codes[b:b + 1].view(torch.float8_e4m3fn).to(DEV), E[b:b + 1].to(DEV), K)
        dy = torch.randn((1, T, N), generator=gen(18)).to(torch.bfloat16).to(DEV)
        dw, _ = fp8_wgrad(x, dy)
        assert torch.equal(dw.double(), ref.outer(ref.value(x), dy.double()))
    ok()


# ---- the FFN ----------------------------------------------------------------------------------------

def ffn(T, D, F, seed):
    g = gen(seed)
    return Fp8PFFN(weight(T, D, F, seed + 1), 0.1 * torch.randn((T, F), generator=g).to(DEV), weight(T, F, D, seed + 2),
                   0.1 * torch.randn((T, D), generator=g).to(DEV))


def code_step(v, scales, cols):
    """Half a step of e4m3 around values v under their exponent bytes."""
    s = ref.pow2(scales[..., :-(-cols // 128)].to(torch.int64) - 127).repeat_interleave(128, -1)[..., :cols]
    return torch.maximum(ref.HALF["e4m3"] * v.abs(), ref.LOWEST["e4m3"] / 2 * s)


FFN_SIZES = [(1, 1, 16, 16), (3, 2, 128, 256), (8, 4, 256, 1024), (40, 3, 208, 416), (100, 2, 384, 640), (129, 1, 256, 272),
             (250, 2, 512, 1536), (300, 3, 144, 400), (1, 32, 256, 512), (16, 1, 128, 400), (17, 3, 272, 128),
             (32, 2, 640, 144), (33, 1, 16, 256), (64, 2, 400, 528), (65, 2, 128, 128), (257, 1, 528, 272)]
# the hidden GELU is within 5e-7 |u| of the exact one (Abramowitz & Stegun 7.1.26: 1.5e-7 in erf; a reciprocal and a
# power of two of 2^-22 each; float32 steps), its derivative within 1e-6 (1 + |u|)
GELU_ERR, GRAD_ERR = 5e-7, 1e-6


@pytest.mark.parametrize("B,T,D,F", FFN_SIZES)
def test_pffn_forward_and_backward_stage_by_stage(B, T, D, F):
    m = ffn(T, D, F, 20)
    X = rows((B, T, D), 23, 0.5).to(torch.bfloat16).to(DEV)
    V, kept = m.forward_train(X, "f32")
    codes, E = ref.quantise(X.cpu(), "e4m3")
    assert torch.equal(kept["x"].codes.view(torch.uint8)[..., :D].cpu(), codes)
    assert torch.equal(kept["x"].scales[..., :E.shape[-1]].cpu(), E)
    w1, w2, xv = ref.weight_value(m.W1), ref.weight_value(m.W2), ref.value(kept["x"])
    u, size = ref.matmul(xv, w1), ref.matmul(xv.abs(), w1.abs())
    u, uerr = u + m.b1.double(), ref.sum_bound(D + 1, size + m.b1.double().abs())
    uv, av = ref.value(kept["u"]), ref.value(kept["a"])
    within(uv, u, uerr + code_step(u.abs() + uerr, kept["u"].scales, F), "kept u")
    aerr = 1.13 * uerr + GELU_ERR * u.abs() + 1e-30
    a = ref.gelu(u)
    within(av, a, aerr + code_step(a.abs() + aerr, kept["a"].scales, F), "kept a")
    for k, v, err in (("u", u, uerr), ("a", a, aerr)):       # the exponents are those of the largest values
        v, err = (torch.nn.functional.pad(z, (0, -F % 128)).reshape(B, T, -1, 128).amax(-1) for z in (v.abs(), err))
        e = kept[k].scales[..., :v.shape[-1]].to(torch.int64) - 127
        assert ((e >= ref.exponent(v - err, "e4m3")) & (e <= ref.exponent(v + err, "e4m3")) | (v <= err)).all(), k
    want, size = ref.matmul(av, w2), ref.matmul(av.abs(), w2.abs())
    within(V, want + m.b2.double(), ref.sum_bound(F + 1, size + m.b2.double().abs()), "V")
    Vs = m.forward(X, "f32")
    assert torch.equal(Vs, V), "serving and training forward differ"
    assert torch.equal(m.forward(X), V.to(torch.bfloat16))

    dV = (torch.randn((B, T, D), generator=gen(24)) * torch.exp(torch.randn((B, T, 1), generator=gen(25)))).to(
        torch.bfloat16).to(DEV)
    dX, g = m.backward(dV, kept, "f32", "f32")
    dv8 = ref.rounded(dV.double())
    da, size = ref.matmul(dv8, w2.transpose(1, 2)), ref.matmul(dv8.abs(), w2.abs().transpose(1, 2))
    slope = ref.gelu_grad(uv)
    du = da * slope
    duerr = ref.sum_bound(D, size) * 1.13 + GRAD_ERR * (1 + uv.abs()) * da.abs()
    half = duerr + ref.HALF_BF16 * (du.abs() + duerr)          # rounded to bf16 for the weight gradient
    dw2, dw2s = ref.outer(av, dV.double()), ref.outer(av.abs(), dV.double().abs())
    within(g["dW2"], dw2, ref.sum_bound(B, dw2s), "dW2")
    within(g["db2"], dV.double().sum(0), ref.sum_bound(B, dV.double().abs().sum(0)), "db2")
    within(g["dW1"], ref.outer(xv, du), ref.sum_bound(B, ref.outer(xv.abs(), du.abs() + half)) + ref.outer(xv.abs(), half),
           "dW1")
    within(g["db1"], du.sum(0), ref.sum_bound(B, (du.abs() + half).sum(0)) + half.sum(0), "db1")
    # dX: dU in 8 bits, each value off by half a step (a largest value at a border may double its block's step)
    step = duerr + 2 * code_step(du.abs() + duerr, _scales(du), F)
    dxw = w1.transpose(1, 2)
    within(dX, ref.matmul(du, dxw),
           ref.matmul(step, dxw.abs()) + ref.sum_bound(F, ref.matmul(du.abs() + step, dxw.abs())), "dX")
    # ... and in norm: half a step is uniform in +-2^-4 |du|, well below 2^-4 of the whole
    off = (dX.double() - ref.matmul(du, dxw)).norm() / ref.matmul(du, dxw).norm()
    near = (dX.double() - ref.matmul(ref.rounded(du), dxw)).norm() / ref.matmul(du, dxw).norm()
    print(f"dX {off:.3g} from the unrounded, {near:.3g} from the rounded gradient")
    assert off <= 2.0 ** -4 and near <= 2.0 ** -8
    # the same again, in the other types
    dXb, gb = m.backward(dV.float(), kept, "bf16", "bf16")
    assert torch.equal(dXb, dX.to(torch.bfloat16))
    for k in g:
        assert gb[k].dtype == torch.bfloat16
        want = g[k].to(torch.bfloat16)
        assert torch.equal(gb[k], want), f"{k}: {int((gb[k] != want).sum())} differ from the rounded float32 gradient"
    none, g2 = m.backward(dV, kept, with_dX=False)
    assert none is None and all(torch.equal(g2[k], g[k]) for k in g)
    ok()


def _scales(x):
    n = x.shape[-1]
    v = torch.nn.functional.pad(x, (0, -n % 128)).reshape(x.shape[:-1] + (-1, 128)).abs().amax(-1)
    return (ref.exponent(v, "e4m3") + 127).to(torch.uint8)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("B,T,K,N", [(1, 8, 2048, 512), (9, 1, 640, 128), (16, 3, 1500, 200), (30, 1, 8192, 100), (48, 2, 4097, 257),
                                     (64, 5, 2500, 384), (64, 38, 2048, 128), (2, 39, 2048, 128), (2, 77, 1024, 128)])
def test_matmul_of_few_samples_and_tiles(B, T, K, N, trans, out):
    """Tiles whose K several thread blocks share: whole and ragged shares, and the counts of tiles around which the rule turns."""
    test_matmul(B, T, K, N, trans, out)


def test_matmul_of_shared_k_is_repeatable():
    x, w = act((40, 8, 2048), 50), weight(8, 2048, 512, 51)
    y = fp8_matmul(x, w, None, "f32")
    for _ in range(20):
        assert torch.equal(fp8_matmul(x, w, None, "f32"), y)
    ok()


@pytest.mark.parametrize("B,T,D,F", [(1, 8, 512, 2048), (12, 4, 1040, 256), (33, 2, 2048, 400), (64, 8, 512, 2048)])
def test_pffn_of_few_samples_and_tiles(B, T, D, F):
    test_pffn_forward_and_backward_stage_by_stage(B, T, D, F)


@pytest.mark.parametrize("B", [6, 40, 300])
def test_pffn_with_hidden_values_of_any_size(B):
    """Hidden pre-activations from 1e-12 to 1e9 (rows of any exponent, far above and below where GELU bends), rows of
    zeros and a row with a NaN: kept values, outputs and gradients follow the formulas, and the NaN stays in its row."""
    T, D, F = 2, 128, 384
    m = ffn(T, D, F, 70)
    m.b1.zero_()
    size = torch.logspace(-12, 9, B).reshape(B, 1, 1)
    X = (rows((B, T, D), 73, 0.0) * size).to(DEV)
    X[2] = 0
    X[1, 1, 5] = float("nan")
    V, kept = m.forward_train(X, "f32")
    dV = rows((B, T, D), 74, 0.5).to(torch.bfloat16).to(DEV)
    dX, _ = m.backward(dV, kept, "f32")
    bad = torch.zeros((B, T, 1), dtype=torch.bool, device=DEV)
    bad[1, 1] = True
    assert torch.equal(V.isnan(), bad.expand(B, T, D)) and torch.equal(dX.isnan(), bad.expand(B, T, D))
    fine = ~bad[..., 0]
    xv, uv, av = (ref.value(kept[k]) for k in "xua")
    w1, w2 = ref.weight_value(m.W1), ref.weight_value(m.W2)
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    xv = torch.where(bad, zero, xv)
    u, us = ref.matmul(xv, w1), ref.matmul(xv.abs(), w1.abs())
    uerr = ref.sum_bound(D, us)
    within(uv[fine], u[fine], (uerr + code_step(u.abs() + uerr, kept["u"].scales, F))[fine], "kept u")
    a, aerr = ref.gelu(u), 1.13 * uerr + GELU_ERR * u.abs() + 1e-30
    within(av[fine], a[fine], (aerr + code_step(a.abs() + aerr, kept["a"].scales, F))[fine], "kept a")
    av, uv = torch.where(bad, zero, av), torch.where(bad, zero, uv)
    want, vs = ref.matmul(av, w2), ref.matmul(av.abs(), w2.abs())
    within(V[fine], (want + m.b2.double())[fine], ref.sum_bound(F + 1, vs + m.b2.double().abs())[fine], "V")
    dv8 = ref.rounded(dV.double())
    da, das = ref.matmul(dv8, w2.transpose(1, 2)), ref.matmul(dv8.abs(), w2.abs().transpose(1, 2))
    # beyond |u| = 10 the derivative is 0 or 1 to 1e-21: its formula in float64 would be inf * 0 far out
    slope = ref.gelu_grad(uv.clamp(-30, 30))
    du, duerr = da * slope, ref.sum_bound(D, das) * 1.13 + GRAD_ERR * (1 + uv.abs().clamp(max=30)) * da.abs()
    step = duerr + 2 * code_step(du.abs() + duerr, _scales(du), F)
    dxw = w1.transpose(1, 2)
    tol = ref.matmul(step, dxw.abs()) + ref.sum_bound(F, ref.matmul(du.abs() + step, dxw.abs()))
    within(dX[fine], ref.matmul(du, dxw)[fine], tol[fine], "dX")
    ok()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("B,T,K,N", [(130, 64, 200, 257), (257, 40, 1000, 130), (333, 20, 272, 520), (513, 31, 128, 264),
                                     (1000, 76, 96, 16)])
def test_matmul_of_many_tiles(B, T, K, N, trans, out):
    """More samples than are streamed past the weights, in more tiles than thread blocks fit on the device at once."""
    test_matmul(B, T, K, N, trans, out)


def test_matmul_of_many_tiles_applies_every_exponent_and_keeps_nan():
    B, T, K, N = 2500, 2, 520, 400
    g = gen(52)
    one = torch.ones(1).to(torch.float8_e4m3fn).view(torch.uint8).item()
    E = torch.randint(125, 130, (B, T, 8), generator=g, dtype=torch.uint8)
    Ew = torch.randint(125, 130, (T, 5, 4), generator=g, dtype=torch.uint8)
    x = Fp8Tensor(torch.full((B, T, 528), one, dtype=torch.uint8).view(torch.float8_e4m3fn).to(DEV), E.to(DEV), K)
    w = Fp8Tensor(torch.full((T, K, N), one, dtype=torch.uint8).view(torch.float8_e4m3fn).to(DEV), Ew.to(DEV), N)
    assert torch.equal(fp8_matmul(x, w, None, "f32").double(), ref.matmul(ref.value(x), ref.weight_value(w)))
    test_matmul_keeps_nan_in_its_row_and_reads_no_padding(5000)


@pytest.mark.parametrize("B,T,D,F", [(300, 64, 128, 256), (257, 80, 80, 272), (513, 32, 160, 144)])
def test_pffn_of_many_tiles(B, T, D, F):
    test_pffn_forward_and_backward_stage_by_stage(B, T, D, F)


def test_pffn_of_many_tiles_with_hidden_values_of_any_size():
    test_pffn_with_hidden_values_of_any_size(9800)


def test_the_example_learns():
    from examples.pffn_8bit import train
    r = train(B=300, T=4, D=128, k=2, steps=60)
    assert r["last"] < 0.5 * r["first"], r
    assert r["kept_bytes"] < 0.52 * r["bytes_in_16_bits"]


def test_pffn_gradients_against_differences():
    """dL/dp along random directions for L = sum(R * V): central differences of the unrounded float64 FFN (same 8-bit
    weights).  The 8-bit activations put V and the gradients off by independent half steps, at most 2^-4 of each
    factor: the directional derivatives agree to 2 * 2^-4."""
    B, T, D, F = 64, 2, 256, 512
    m = ffn(T, D, F, 30)
    X = rows((B, T, D), 33, 0.3).to(torch.bfloat16).to(DEV)
    R = torch.randn((B, T, D), generator=gen(34)).to(torch.bfloat16).to(DEV)
    _, kept = m.forward_train(X)
    dX, g = m.backward(R, kept, "f32", "f32")
    p = {"X": X.double(), "W1": ref.weight_value(m.W1), "b1": m.b1.double(), "W2": ref.weight_value(m.W2), "b2": m.b2.double()}

    def loss(q):
        return (R.double() * (ref.matmul(ref.gelu(ref.matmul(q["X"], q["W1"]) + q["b1"]), q["W2"]) + q["b2"])).sum()

    for name, grad in (("X", dX), ("W1", g["dW1"]), ("b1", g["db1"]), ("W2", g["dW2"]), ("b2", g["db2"])):
        d = grad.double() / grad.double().norm()               # the steepest direction, where the derivative is large
        h = 1e-4
        up, down = ({**p, name: p[name] + s * h * d} for s in (1, -1))
        diff, have = (loss(up) - loss(down)) / (2 * h), (grad.double() * d).sum()
        print(f"{name}: difference {diff:.6g}, gradient {have:.6g}")
        assert abs(diff - have) <= 2 * 2.0 ** -4 * abs(diff), name


def test_pffn_takes_plain_weights_and_refuses_what_does_not_fit():
    T, D, F = 2, 64, 128
    g = gen(40)
    W1, W2 = (torch.randn(s, generator=g).to(torch.bfloat16).to(DEV) for s in ((T, D, F), (T, F, D)))
    b1, b2 = torch.zeros((T, F), device=DEV), torch.zeros((T, D), device=DEV)
    m = Fp8PFFN(W1, b1, W2, b2)
    n = Fp8PFFN(fp8_quantize_weight(W1), b1, fp8_quantize_weight(W2), b2)
    X = rows((5, T, D), 41, 0.5).to(DEV)
    V, kept = m.forward_train(X)
    assert torch.equal(V, n.forward(X))
    for bad in (X[..., :32], X[:, :1], X.half(), X[0]):
        with pytest.raises(ValueError):
            m.forward(bad)
    with pytest.raises(ValueError):
        m.forward(X.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        m.backward(X[:4], kept)
    with pytest.raises(ValueError):
        m.backward(X, {**kept, "u": kept["x"]})
    with pytest.raises(_lib.RankMixerError):
        m.forward(X[:0])
    with pytest.raises(ValueError):
        Fp8PFFN(W1, b2, W2, b1)
    with pytest.raises(_lib.RankMixerError):                  # D not a multiple of 16
        Fp8PFFN(W1[:, :40].contiguous(), b1, W2[..., :40].contiguous(), b2[:, :40]).forward(X[..., :40].contiguous())
    ok()


# ---- how they are run --------------------------------------------------------------------------------

@pytest.mark.parametrize("B", [2, 70, 300])
def test_calls_are_repeatable_on_any_stream_and_in_graphs(B):
    T, D, F = 3, 256, 512
    m = ffn(T, D, F, 50)
    X = rows((B, T, D), 53, 0.5).to(torch.bfloat16).to(DEV)
    dV = rows((B, T, D), 54, 0.5).to(torch.bfloat16).to(DEV)

    def step():
        V, kept = m.forward_train(X)
        dX, g = m.backward(dV, kept)
        dW, db = fp8_wgrad(kept["a"], dV)
        return [V, dX, *g.values(), dW, db, m.forward(X), fp8_matmul(kept["x"], m.W1, m.b1), fp8_dequantize(kept["u"])]

    first = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        other = step()
        assert api.fp8_sync_status() == _lib.RM_OK
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    X2, dV2 = rows((B, T, D), 55, 0.5).to(torch.bfloat16).to(DEV), rows((B, T, D), 56, 0.5).to(torch.bfloat16).to(DEV)
    X.copy_(X2)
    dV.copy_(dV2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))
    ok()


def test_two_streams_do_not_share_anything():
    T, D, F = 2, 256, 1024
    m = ffn(T, D, F, 60)
    Xs = [rows((150 + 40 * i, T, D), 63 + i, 0.5).to(torch.bfloat16).to(DEV) for i in range(4)]
    want = [m.forward(X) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = []
    for s, X in zip(streams, Xs):
        with torch.cuda.stream(s):
            got.append([m.forward(X) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(v, w) for vs, w in zip(got, want) for v in vs)
    ok()
