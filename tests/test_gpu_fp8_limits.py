"""GPU tests of the 8-bit operators where their ranges end: GELU's far tail, sums of many samples, what is shared
between streams, and forms of the arguments that the products of ordinary layers do not take."""
from __future__ import annotations

import math
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300.api import (Fp8PFFN, Fp8Tensor, fp8_matmul, fp8_quantize, fp8_quantize_weight,
                                                     fp8_sync_status, fp8_wgrad)
from tests import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# ---- weight gradients that are joined from chunks -----------------------------------------------------

def wgrad_into(x, dy, dtype, with_db=True, fill=float("nan")):
    """The C entry, into buffers that hold `fill`: (dW, db)."""
    (B, T, K), N = x.shape, dy.shape[-1]
    tdt, code = (torch.float32, _lib.RM_F32) if dtype == "f32" else (torch.bfloat16, _lib.RM_BF16)
    dw, db = (torch.full(s, fill, dtype=tdt, device=DEV) for s in ((T, K, N), (T, N)))
    _lib.rm_fp8_wgrad(x.c, dy.data_ptr(), dw.data_ptr(), db.data_ptr() if with_db else None, code, B, T, K, N,
                      torch.cuda.current_stream().cuda_stream)
    return dw, db


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,K,N", [(2049, 2, 272, 520), (4161, 3, 130, 264), (9000, 1, 1001, 40), (4096, 40, 500, 776),
                                     (6145, 80, 128, 136)])
def test_wgrad_of_several_chunks(B, T, K, N, dtype):
    """Elementwise as for one chunk (float32 additions of B exact products), the buffers full of NaN and then of ones
    before the call: the first chunk overwrites, the others add once."""
    x = fp8_quantize(torch.randn((B, T, K), generator=torch.Generator(device=DEV).manual_seed(88), device=DEV))
    dy = torch.randn((B, T, N), generator=torch.Generator(device=DEV).manual_seed(89), device=DEV).to(torch.bfloat16)
    xv, yv = ref.value(x), dy.double()
    dw, db = wgrad_into(x, dy, dtype)
    again = wgrad_into(x, dy, dtype, fill=1.0)
    assert torch.equal(again[0], dw) and torch.equal(again[1], db)
    for got, want, size, what in ((dw, ref.outer(xv, yv), ref.outer(xv.abs(), yv.abs()), "dW"),
                                  (db, yv.sum(0), yv.abs().sum(0), "db")):
        tol = ref.sum_bound(B, size)
        if dtype == "bf16":
            tol = tol + ref.HALF_BF16 * (want.abs() + tol)
        within(got, want, tol, f"{what} {dtype}")
    if dtype == "f32":
        # a lost or doubled chunk is off by about 1 / sqrt(chunks) in norm; the sums lose at most 2^-17 (a chunk of terms
        # of one sign) of the magnitudes' sum, in norm at most sqrt(B) times the gradient of independent samples
        off = ((dw.double() - ref.outer(xv, yv)).norm() / ref.outer(xv, yv).norm()).item()
        assert off <= 2.0 ** -17 * math.sqrt(B), off
    ok()


@pytest.mark.parametrize("B", [3, 700, 5000])
def test_wgrad_without_the_bias_gradient(B):
    T, K, N = 3, 400, 776
    x = fp8_quantize(torch.randn((B, T, K), generator=gen(90)).to(DEV))
    dy = torch.randn((B, T, N), generator=gen(91)).to(torch.bfloat16).to(DEV)
    for dtype in ("f32", "bf16"):
        dw, db = wgrad_into(x, dy, dtype, with_db=False)
        assert torch.equal(dw, wgrad_into(x, dy, dtype)[0]) and db.isnan().all()
    ok()


# ---- forms of the arguments -----------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,trans", [("e5m2", False), ("e4m3", True)])
@pytest.mark.parametrize("B,T,K,N", [(1, 3, 200, 72), (20, 1, 2048, 130), (100, 2, 257, 129), (333, 20, 272, 520)])
def test_either_format_in_either_direction(B, T, K, N, fmt, trans):
    x = fp8_quantize(torch.randn((B, T, K), generator=gen(92)).to(DEV), fmt)
    w = fp8_quantize_weight(torch.randn((T, N, K) if trans else (T, K, N), generator=gen(93)).to(DEV))
    wv = ref.weight_value(w)
    xv, wv = ref.value(x), wv.transpose(1, 2) if trans else wv
    within(fp8_matmul(x, w, None, "f32", trans), ref.matmul(xv, wv), ref.sum_bound(K, ref.matmul(xv.abs(), wv.abs())),
           f"{fmt} trans={trans}")
    ok()


@pytest.mark.parametrize("C,extra", [(200, 48), (1003, 16), (128, 400)])
def test_rows_longer_than_their_columns(C, extra):
    """Code, scale and value rows with room behind them, which stays as it is; products and gradients read past it."""
    B, T, N = 140, 2, 136
    ld, lds = (C + 15) // 16 * 16 + extra, (C + 511) // 512 * 4 + 8
    v = torch.randn((B, T, C), generator=gen(94)).to(DEV)
    codes = torch.full((B, T, ld), 0x7f, dtype=torch.uint8, device=DEV)
    scales = torch.full((B, T, lds), 255, dtype=torch.uint8, device=DEV)
    q = Fp8Tensor(codes.view(torch.float8_e4m3fn), scales, C)
    s = torch.cuda.current_stream().cuda_stream
    _lib.rm_fp8_quantize(v.data_ptr(), _lib.RM_F32, B * T, C, C, q.c, s)
    plain = fp8_quantize(v)
    nb = (C + 127) // 128
    assert torch.equal(codes[..., :C], plain.codes.view(torch.uint8)[..., :C])
    assert torch.equal(scales[..., :nb], plain.scales[..., :nb])
    assert (codes[..., (C + 15) // 16 * 16:] == 0x7f).all() and (scales[..., nb:] == 255).all()
    for dt, code in ((torch.float32, _lib.RM_F32), (torch.bfloat16, _lib.RM_BF16)):
        for ldy in (C, C + 1, C + 24):
            y = torch.full((B * T, ldy), 7.0, dtype=dt, device=DEV)
            _lib.rm_fp8_dequantize(q.c, B * T, C, y.data_ptr(), code, ldy, s)
            assert torch.equal(y[:, :C].double().reshape(B, T, C), ref.value(plain)) and (y[:, C:] == 7).all()
    w = fp8_quantize_weight(torch.randn((T, C, N), generator=gen(95)).to(DEV))
    for b in (7, B):
        part = Fp8Tensor(q.codes[:b], q.scales[:b], C)
        whole = Fp8Tensor(plain.codes[:b], plain.scales[:b], C)
        assert torch.equal(fp8_matmul(part, w, None, "f32"), fp8_matmul(whole, w, None, "f32"))
        dy = torch.randn((b, T, N), generator=gen(96)).to(torch.bfloat16).to(DEV)
        assert all(torch.equal(a, c) for a, c in zip(fp8_wgrad(part, dy), fp8_wgrad(whole, dy)))
    ok()


# ---- what the streams of a device share -----------------------------------------------------------------

def in_child(body):
    """Run `body` in a process of its own: its errors and first calls are not this process's."""
    code = "import torch\nfrom rankmixer_feature_interaction_gb300 import _lib, api\n" + textwrap.dedent(body)
    env = {**os.environ, "PYTHONPATH": ROOT}
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_wait_that_ran_out_is_reported_to_every_stream():
    """A wait with a short limit runs out on one stream.  Whichever stream is asked first, the other one's report is
    not lost; each is told once, and later calls are right."""
    in_child("""
        g = torch.Generator(device="cuda").manual_seed(1)
        x = api.fp8_quantize(torch.randn((200, 2, 256), generator=g, device="cuda"))
        w = api.fp8_quantize_weight(torch.randn((2, 256, 512), generator=g, device="cuda"))
        want = api.fp8_matmul(x, w)
        assert api.fp8_sync_status() == _lib.RM_OK
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for n in range(2):
            _lib.rm_debug_fp8_wait_timeout(2000, b.cuda_stream)
            torch.cuda.synchronize()
            for s in (a, b, torch.cuda.current_stream()):
                with torch.cuda.stream(s):
                    first, then, y = api.fp8_sync_status(), api.fp8_sync_status(), api.fp8_matmul(x, w)
                    last = api.fp8_sync_status()
                assert (first, then, last) == (_lib.RM_ERR_TIMEOUT, _lib.RM_OK, _lib.RM_OK), (n, first, then, last)
                assert torch.equal(y, want)
        new = torch.cuda.Stream(priority=-1)           # never asked before: told of what happened before, once
        with torch.cuda.stream(new):
            assert api.fp8_sync_status() == _lib.RM_ERR_TIMEOUT and api.fp8_sync_status() == _lib.RM_OK
    """)


def test_the_wait_hook_refuses_other_limits():
    for us in (0, -1, 10000001):
        with pytest.raises(_lib.RankMixerError):
            _lib.rm_debug_fp8_wait_timeout(us, 0)


@pytest.mark.parametrize("first", ["pass", "api.fp8_quantize(X)", "api.fp8_quantize_weight(W)", "api.fp8_dequantize(x)"])
def test_first_calls_may_be_captured(first):
    """Products and gradients captured at their first call, after another 8-bit call or none."""
    in_child(f"""
        X, W = torch.ones((40, 2, 256), device="cuda"), torch.ones((2, 256, 256), device="cuda")
        dY = torch.ones((40, 2, 256), device="cuda").to(torch.bfloat16)
        def ones(shape, blocks):
            return api.Fp8Tensor(torch.ones(shape, device="cuda").to(torch.float8_e4m3fn),
                                 torch.full(blocks, 127, dtype=torch.uint8, device="cuda"), shape[-1])
        x, w = ones((40, 2, 256), (40, 2, 4)), ones((2, 256, 256), (2, 2, 4))
        {first}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, (dw, db) = api.fp8_matmul(x, w), api.fp8_wgrad(x, dY)
        graph.replay()
        torch.cuda.synchronize()
        assert (y == 256).all() and (dw == 40).all() and (db == 40).all()
        assert api.fp8_sync_status() == _lib.RM_OK
    """)


# ---- how few tiles share their sums ---------------------------------------------------------------------

def graph_us(call, n=50, reps=7):
    """Device time of one call among others, in a graph (the best of some replays)."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    best = math.inf
    for _ in range(reps):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


@pytest.mark.parametrize("B,K", [(8, 2048), (8, 4096), (40, 2048)])
def test_fewer_tiles_do_not_take_longer_than_more(B, K):
    """One tile a token.  K is shared by clusters of thread blocks only where all of them are resident at once: with a
    second round of clusters 38 tiles took 1.5 times as long as 39 by clusters of two."""
    us = {}
    for T in (30, 34, 36, 37, 38, 39, 44, 72, 76, 77):
        x = fp8_quantize(torch.randn((B, T, K), generator=torch.Generator(device=DEV).manual_seed(97), device=DEV))
        w = fp8_quantize_weight(torch.randn((T, K, 128), generator=torch.Generator(device=DEV).manual_seed(98), device=DEV))
        us[T] = graph_us(lambda: fp8_matmul(x, w))
    print(" ".join(f"{t}: {v:.2f}" for t, v in us.items()))
    for few in us:
        for more in us:
            if few < more:
                assert us[few] <= 1.25 * us[more], (few, more, us)
    ok()
