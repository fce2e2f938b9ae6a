"""GPU tests of the 4-bit operators and of the experts' rows where their ranges end: GELU's far tail, the longest sums,
offsets past 32 bits, rows and weights with room behind them, graphs, streams, and the bounds-checked build."""
from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300.api import (Fp4MoE, Fp4PFFN, Fp4Tensor, expert_combine, expert_combine_backward,
                                                     expert_gather, expert_gather_backward, expert_sort, fp4_dequantize,
                                                     fp4_expert_gather, fp4_expert_matmul, fp4_matmul, fp4_quantize, fp4_quantize_weight)
from tests import fp4_reference as ref
from tests.test_gpu_experts import gates
from tests.test_gpu_fp4 import DEV, gen, layer, ok, rows, weight, within
from tests.test_nvtx_ranges import ranges

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def stream():
    return torch.cuda.current_stream().cuda_stream


def in_child(body):
    """Run `body` in a process of its own: its first calls are not this process's."""
    code = "import torch\nfrom rankmixer_feature_interaction_gb300 import _lib, api\n" + textwrap.dedent(body)
    env = {**os.environ, "PYTHONPATH": ROOT}
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


# ---- hidden values and sums ---------------------------------------------------------------------------

RANGES = [(-7, -6), (-9, -6), (-12.5, -10), (-5.5, -4.5), (-20, -13), (-1e4, -50), (-1e30, -1e28), (-6.5, 6.5), (-3, -2),
          (6, 50), (-3.3e38, -3e38), (-0.01, 0.01), (-8, -7), (3e30, 3e38)]


@pytest.mark.parametrize("B", [1, 20, 40, 100, 300])
def test_hidden_values_of_blocks_far_from_zero(B):
    """The input is zero, so the hidden pre-activations are the biases exactly, and W2 is the identity, so the output is
    the hidden activation as it was rounded.  Gelu is within 3.5e-7 |u| (and zero below -12.85, where it is less than that),
    and besides within 1.6% of its tail: 1.5% of the fit and 8 float32 steps of a logarithm."""
    T, D = 28, 256
    lo, hi = (torch.tensor([RANGES[i % len(RANGES)][k] for i in range(8 * T)], dtype=torch.float64) for k in (0, 1))
    r = torch.rand((8 * T, 32), generator=gen(80), dtype=torch.float64)
    b1 = (lo[:, None] + (hi - lo)[:, None] * r).float().reshape(T, D).to(DEV)
    eye = torch.eye(D).repeat(T, 1, 1).to(DEV)
    m = Fp4PFFN(torch.randn((T, D, D), generator=gen(81)).to(DEV), b1, eye, torch.zeros((T, D), device=DEV))
    assert torch.equal(ref.weight_value(m.W2).float(), eye)
    V = m.forward(torch.zeros((B, T, D), device=DEV), "f32")
    u = b1.double()
    a, tail = ref.gelu(u), 0.5 * torch.special.erfc(u.abs() / 2 ** 0.5)
    err = u.abs() * torch.minimum(torch.full_like(u, 3.5e-7), 0.016 * tail) + ref.UNIT_F32 * a.abs()
    err = torch.where(u < -12.85, a.abs(), err)
    # a value above 7/2 2^126 rounds to 4 2^126 = 2^128, which is an infinity in float32
    low, high = (v.float() for v in ref.rounded_between(a, err)[1:])
    assert ((V >= low) & (V <= high)).all(), int(((V < low) | (V > high)).sum())
    ok()


def test_the_largest_values():
    """Above 7/2 2^126 the nearest code is 4 2^126 = 2^128: an infinity where it is read back."""
    x = torch.tensor([3.4e38, 2.98e38, 2.97e38, -3.4e38, 1.0], device=DEV)
    q = fp4_quantize(x)
    assert q.scales[0] == 253
    for out in ("f32", "bf16"):
        assert fp4_dequantize(q, out).double().tolist() == [torch.inf, torch.inf, 3 * 2.0 ** 126, -torch.inf, 0.0]


@pytest.mark.parametrize("B", [1, 40, 300])
def test_products_of_the_longest_sums(B):
    """Terms of one sign, K = 2^19: K / 64 instructions, each loses at most a unit in the last place (2^-23) of what it
    adds and of a running sum that is half the final one on average, in all K / 64 * 2^-23 = 2^-10."""
    K, N = 1 << 19, 16
    positive = lambda *s: torch.rand(s, generator=torch.Generator(device=DEV).manual_seed(83), device=DEV) + 0.3   # noqa: E731
    x, w = fp4_quantize(positive(B, 1, K)), fp4_quantize_weight(positive(1, K, N))
    want = ref.matmul(ref.value(x), ref.weight_value(w))
    within(fp4_matmul(x, w, None, "f32"), want, 2.0 ** -10 * want, "K = 2^19")
    ok()


# ---- past 32 bits ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("B,T,N", [(128, 1000, 20480), (4096, 32, 20480)])
def test_products_past_32_bits(B, T, N):
    """More than 2^31 outputs: the last rows and some others are what smaller calls give."""
    K = 32
    x = fp4_quantize(torch.randn((B, T, K), generator=torch.Generator(device=DEV).manual_seed(84), device=DEV))
    w = fp4_quantize_weight(torch.randn((T, K, N), generator=torch.Generator(device=DEV).manual_seed(85), device=DEV))
    y = fp4_matmul(x, w)
    assert y.numel() > 1 << 31
    xv = ref.value(x)
    for b, t in ((0, 0), (B - 1, T - 1), (B // 2, T - 1), (B - 1, 0)):
        part = Fp4Tensor(w.codes[t:t + 1].contiguous(), w.scales[t:t + 1].contiguous(), K, weight=True)
        want = xv[b, t] @ ref.weight_value(part)[0]
        size = xv[b, t].abs() @ ref.weight_value(part)[0].abs()
        tol = ref.sum_bound(K, size)
        within(y[b, t], want, tol + (want.abs() + tol) * ref.HALF_BF16, f"row {b} {t}")
    ok()


def test_rows_past_32_bits():
    """More than 2^31 values in the sorted rows."""
    B, T, E, D = 4096, 32, 8, 2056
    G = torch.ones((B, T, E), device=DEV)
    r = expert_sort(G)
    n = r.count()
    assert n == B * T * E and n * D > 1 << 31
    X = torch.randn((B, T, D), generator=torch.Generator(device=DEV).manual_seed(86), device=DEV).to(torch.bfloat16)
    Xs = expert_gather(X, r)
    for b, t, e in ((0, 0, 0), (B - 1, T - 1, E - 1), (17, 31, 7), (B - 1, 0, 3)):
        assert int(r.slot[b, t, e]) == (t * E + e) * B + b
        assert torch.equal(Xs[(t * E + e) * B + b], X[b, t])
    V = expert_combine(Xs, r, G)
    assert torch.equal(V[-3:], X[-3:] * 8) and torch.equal(V[:3], X[:3] * 8)
    dX = expert_gather_backward(Xs, r)
    assert torch.equal(dX[-3:], X[-3:] * 8)
    del V, dX
    dY, dG = expert_combine_backward(X, Xs, r, G)
    assert torch.equal(dY[-1], X[-1, -1]) and torch.equal(dY[0], X[0, 0])
    want = (X[-1, -1].double() ** 2).sum()
    assert abs(dG[-1, -1, -1].double() - want) <= ref.sum_bound(D, want)
    ok()


def test_the_longest_rows():
    """One row of nearly 2^31 values, to two experts and back: steps end past 2^31."""
    D = 2 ** 31 - 513
    G = torch.tensor([[[0.5, 2.0]]], device=DEV)
    r = expert_sort(G)
    X = torch.zeros((1, 1, D), dtype=torch.bfloat16, device=DEV)
    at = [0, 1, 12345, 2 ** 30, D - 1200, D - 2, D - 1]
    value = torch.tensor([1.0, -2.0, 3.0, 5.0, -7.0, 11.0, 13.0])
    X[0, 0, at] = value.to(DEV, torch.bfloat16)
    Xs = expert_gather(X, r, 2)
    assert torch.equal(Xs[0], X[0, 0]) and torch.equal(Xs[1], X[0, 0])
    V = expert_combine(Xs, r, G)
    assert V[0, 0, at].float().cpu().tolist() == (2.5 * value).tolist() and int(V.count_nonzero()) == len(at)
    del V
    dY, dG = expert_combine_backward(X, Xs, r, G)
    assert dG.flatten().tolist() == [(value ** 2).sum().item()] * 2
    for e, g in enumerate((0.5, 2.0)):
        assert dY[e, at].float().cpu().tolist() == (g * value).tolist() and int(dY[e].count_nonzero()) == len(at)
    ok()


@pytest.mark.parametrize("D", [2 ** 31 - 512, 2 ** 31 - 513])
def test_the_longest_rows_in_4_bits(D):
    at = torch.tensor([0, 1, 12345, 2 ** 30, D - 1200, D - 2, D - 1])
    value = torch.tensor([1.0, -2.0, 3.0, 6.0, -1.5, 4.0, 0.5], dtype=torch.bfloat16)     # 4-bit numbers in their blocks
    X = torch.zeros((1, 1, D), dtype=torch.bfloat16, device=DEV)
    X[0, 0, at.to(DEV)] = value.to(DEV)
    q = fp4_quantize(X)
    y = fp4_dequantize(q)
    assert y[0, 0, at.to(DEV)].tolist() == value.tolist() and int(y.count_nonzero()) == len(at)
    del y
    r = expert_sort(torch.ones((1, 1, 2), device=DEV))
    x = fp4_expert_gather(X, r, 2)
    for i in range(2):
        assert torch.equal(x.codes[i], q.codes[0, 0]) and torch.equal(x.scales[i, :-(-D // 32)], q.scales[0, 0, :-(-D // 32)])
    ok()


def test_experts_products_past_32_bits():
    """More than 2^31 outputs of sorted rows."""
    B, T, E, K, N = 4096, 32, 8, 64, 2304
    r = expert_sort(torch.ones((B, T, E), device=DEV))
    X = torch.randn((B, T, K), generator=torch.Generator(device=DEV).manual_seed(87), device=DEV)
    w = fp4_quantize_weight(torch.randn((T, E, K, N), generator=torch.Generator(device=DEV).manual_seed(88), device=DEV))
    x = fp4_expert_gather(X, r)
    y = fp4_expert_matmul(x, w, r)
    assert y.numel() > 1 << 31
    wv = ref.weight_value(w)
    for b, t, e in ((0, 0, 0), (B - 1, T - 1, E - 1), (5, 31, 7)):
        a = ref.value(fp4_quantize(X[b, t]))
        want, tol = a @ wv[t, e], ref.sum_bound(K, a.abs() @ wv[t, e].abs())
        within(y[(t * E + e) * B + b], want, tol + (want.abs() + tol) * ref.HALF_BF16, f"{b} {t} {e}")
    ok()


# ---- forms of the arguments -----------------------------------------------------------------------------

@pytest.mark.parametrize("B", [7, 140, 300])
def test_rows_and_weights_longer_than_their_columns(B):
    """Room behind the codes of rows and weights and behind the scales of rows stays as it is; products read past it."""
    T, C, N = 2, 200, 136
    v = torch.randn((B, T, C), generator=gen(94)).to(DEV)
    codes = torch.full((B, T, 160), 0x77, dtype=torch.uint8, device=DEV)
    scales = torch.full((B, T, 32), 255, dtype=torch.uint8, device=DEV)
    q, plain = Fp4Tensor(codes, scales, C), fp4_quantize(v)
    _lib.rm_fp4_quantize(v.data_ptr(), _lib.RM_F32, B * T, C, C, q.c, stream())
    assert torch.equal(codes[..., :112], plain.codes) and (codes[..., 112:] == 0x77).all()
    assert torch.equal(scales[..., :7], plain.scales[..., :7]) and (scales[..., 7:] == 255).all()
    for dt, code in ((torch.float32, _lib.RM_F32), (torch.bfloat16, _lib.RM_BF16)):
        for ldy in (C, C + 1, C + 24):
            y = torch.full((B * T, ldy), 7.0, dtype=dt, device=DEV)
            _lib.rm_fp4_dequantize(q.c, B * T, C, y.data_ptr(), code, ldy, stream())
            assert torch.equal(y[:, :C].double().reshape(B, T, C), ref.value(plain)) and (y[:, C:] == 7).all()
    W = torch.randn((T, C, N), generator=gen(95)).to(DEV)
    w = fp4_quantize_weight(W)
    wide = torch.full((T, N, 144), 0x77, dtype=torch.uint8, device=DEV)
    w2 = Fp4Tensor(wide, torch.zeros_like(w.scales), C, weight=True)
    _lib.rm_fp4_quantize_weight(W.data_ptr(), _lib.RM_F32, T, C, N, w2.c, stream())
    assert torch.equal(wide[..., :112], w.codes) and (wide[..., 112:] == 0x77).all() and torch.equal(w2.scales, w.scales)
    want = fp4_matmul(plain, w, None, "f32")
    assert torch.equal(fp4_matmul(q, w2, None, "f32"), want)
    # an output that is 16-byte aligned and no more
    buf = torch.empty(B * T * N + 4, device=DEV)
    _lib.rm_fp4_matmul(q.c, w.c, None, buf[4:].data_ptr(), _lib.RM_F32, B, T, C, N, stream())
    assert torch.equal(buf[4:].view(B, T, N), want)
    ok()


def test_the_python_calls_refuse_what_does_not_fit():
    x, w = fp4_quantize(torch.ones((3, 2, 64), device=DEV)), weight(2, 64, 32, 1)
    G = torch.ones((3, 2, 4), device=DEV)
    r = expert_sort(G)
    Xs = expert_gather(torch.ones((3, 2, 8), device=DEV), r)
    bad = [lambda: fp4_matmul(x, weight(2, 96, 32, 1)), lambda: fp4_matmul(x, weight(3, 64, 32, 1)), lambda: fp4_matmul(w, x),
           lambda: fp4_matmul(x, w, torch.ones((2, 31), device=DEV)), lambda: fp4_matmul(x, w, torch.ones((2, 32))),
           lambda: fp4_matmul(x, w, torch.ones((2, 32), device=DEV).half()),
           lambda: fp4_matmul(x, w, torch.ones((32, 2), device=DEV).T), lambda: expert_sort(G.double()),
           lambda: expert_sort(G[0]), lambda: expert_sort(G.transpose(0, 1)),
           lambda: expert_gather(torch.ones((4, 2, 8), device=DEV), r), lambda: expert_gather(torch.ones((3, 2), device=DEV), r),
           lambda: expert_gather(torch.ones((3, 2, 8), device=DEV).half(), r),
           lambda: expert_gather(torch.ones((3, 2, 8), device=DEV), r, -1),
           lambda: expert_gather(torch.ones((3, 2, 8)), r), lambda: expert_gather(torch.ones((2, 3, 8), device=DEV).transpose(0, 1), r),
           lambda: expert_combine(Xs, r, G[:, :, :3]), lambda: expert_combine(Xs, r, G.double()), lambda: expert_combine(Xs[0], r, G),
           lambda: expert_combine(Xs.cpu(), r, G), lambda: expert_combine(Xs, r, G.cpu()),
           lambda: expert_combine_backward(torch.ones((3, 2, 9), device=DEV), Xs, r, G),
           lambda: expert_combine_backward(torch.ones((3, 2, 8), device=DEV).to(torch.bfloat16), Xs, r, G),
           lambda: expert_combine_backward(torch.ones((1, 2, 8), device=DEV).expand(3, 2, 8), Xs, r, G),
           lambda: fp4_expert_matmul(x, fp4_quantize_weight(torch.ones((2, 4, 64, 8), device=DEV)), r),
           lambda: fp4_expert_matmul(fp4_quantize(torch.ones((24, 64), device=DEV)),
                                     fp4_quantize_weight(torch.ones((2, 3, 64, 8), device=DEV)), r)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: expert_sort(G[:0]),
                 lambda: fp4_quantize_weight(torch.ones((2, 0, 8), device=DEV))):
        with pytest.raises(_lib.RankMixerError):
            call()
    f = Fp4PFFN(*layer((2,), 64, 32, 2))
    m = Fp4MoE(*layer((2, 4), 64, 32, 3))
    X = torch.ones((3, 2, 64), device=DEV)
    for call in (lambda: f.forward(X[:, :1]), lambda: f.forward(X.half()), lambda: f.forward(X.cpu()), lambda: m.forward(X, G[:2]),
                 lambda: m.forward(X, G.double()), lambda: m.forward(X, G.cpu()), lambda: f.forward(X.expand(3, 2, 64)[..., ::2])):
        with pytest.raises(ValueError):
            call()
    ok()


# ---- graphs and streams -----------------------------------------------------------------------------------

@pytest.mark.parametrize("B", [6, 200])
def test_first_calls_may_be_captured_and_replayed_on_new_inputs(B):
    """The whole set captured at its first call; the replay follows what the inputs hold then: other values, other gates."""
    in_child(f"""
        B, T, E, D, F = {B}, 2, 3, 64, 96
        g = torch.Generator(device="cuda").manual_seed(1)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        X, G, dV = rnd(B, T, D), torch.relu(rnd(B, T, E)), rnd(B, T, D)
        f = api.Fp4PFFN(rnd(T, D, F), rnd(T, F), rnd(T, F, D), rnd(T, D))
        m = api.Fp4MoE(rnd(T, E, D, F), rnd(T, E, F), rnd(T, E, F, D), rnd(T, E, D))
        def step():
            r = api.expert_sort(G)
            Xs = api.expert_gather(X, r)
            V = api.expert_combine(Xs, r, G)
            dY, dG = api.expert_combine_backward(dV, Xs, r, G)
            return V, dG, api.expert_gather_backward(Xs, r), f.forward(X), m.forward(X, G), r.offsets, r.slot
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for n in range(3):
            X.copy_(rnd(B, T, D)), G.copy_(torch.relu(rnd(B, T, E) - n)), dV.copy_(rnd(B, T, D))
            graph.replay()
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), n
        assert api.fp8_sync_status() == _lib.RM_OK
    """)


def test_calls_on_two_streams_at_once():
    B, T, E, D, F = 300, 2, 3, 128, 256
    f, m = Fp4PFFN(*layer((T,), D, F, 4)), Fp4MoE(*layer((T, E), D, F, 5))
    X = [rows((B, T, D), 6 + i).to(DEV) for i in range(2)]
    G = [gates(B, T, E, 0.5, 8 + i).to(DEV) for i in range(2)]

    def step(i):
        r = expert_sort(G[i])
        return f.forward(X[i]), m.forward(X[i], G[i]), expert_combine(expert_gather(X[i], r), r, G[i])
    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(step(i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    ok()


def test_large_launches_on_two_streams_share_the_device():
    """Persistent kernels of two streams, each of which alone fills the device."""
    B, T, K, N = 600, 8, 512, 2048
    x, w = fp4_quantize(rows((B, T, K), 10).to(DEV)), weight(T, K, N, 11)
    y0 = fp4_matmul(x, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(fp4_matmul(x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, y0) for y in got)
    ok()


# ---- ranges and the bounds-checked build -------------------------------------------------------------------

def test_ffns_are_ranged(tmp_path):
    got = ranges(tmp_path, """
        import torch
        from rankmixer_feature_interaction_gb300 import api
        one = lambda *s: torch.ones(s, device="cuda")
        f = api.Fp4PFFN(one(2, 32, 64), one(2, 64), one(2, 64, 32), one(2, 32))
        m = api.Fp4MoE(one(2, 3, 32, 64), one(2, 3, 64), one(2, 3, 64, 32), one(2, 3, 32))
        f.forward(one(5, 2, 32))
        m.forward(one(5, 2, 32), one(5, 2, 3))
    """)
    assert got == ["rm:fp4_quantize_weight"] * 4 + ["rm:fp4_quantize"] + ["rm:fp4_product"] * 2 + \
        ["rm:expert_sort", "rm:fp4_expert_gather", "rm:fp4_product", "rm:fp4_product", "rm:expert_combine"]


CHILD = r"""
import sys, torch
from rankmixer_feature_interaction_gb300 import _lib, api
_lib.load()
maps = open("/proc/self/maps").read()
assert ("librankmixer_debug.so" in maps) == (sys.argv[2] == "debug")
out, g = [], torch.Generator(device="cuda").manual_seed(5)
def rnd(*s): return torch.randn(s, generator=g, device="cuda")
for B, T, K, N in ((1, 8, 2048, 512), (40, 3, 200, 130), (300, 20, 272, 520), (257, 2, 1001, 333)):
    X = rnd(B, T, K)
    q, w = api.fp4_quantize(X), api.fp4_quantize_weight(rnd(T, K, N))
    out += [q.codes, q.scales[..., :(K + 31) // 32], w.codes, w.scales, api.fp4_dequantize(q), api.fp4_dequantize(q, "f32"),
            api.fp4_matmul(q, w, rnd(T, N), "f32"), api.fp4_matmul(q, w)]
for B, T, E, D, F in ((3, 4, 3, 128, 256), (70, 2, 5, 160, 416), (300, 4, 3, 160, 416)):
    f = api.Fp4PFFN(rnd(T, D, F), rnd(T, F), rnd(T, F, D), rnd(T, D))
    m = api.Fp4MoE(rnd(T, E, D, F), rnd(T, E, F), rnd(T, E, F, D), rnd(T, E, D))
    X, G = rnd(B, T, D), torch.relu(rnd(B, T, E))
    r = api.expert_sort(G)
    n = r.count()
    Xs = api.expert_gather(X, r, n)
    out += [f.forward(X), m.forward(X, G), r.offsets, r.source[:n], r.slot, Xs, api.expert_combine(Xs, r, G),
            *api.expert_combine_backward(X, Xs, r, G), api.expert_gather_backward(Xs, r),
            api.fp4_expert_matmul(api.fp4_expert_gather(X, r, n), m.W1, r, m.b1, "f32")]
assert api.fp8_sync_status() == _lib.RM_OK
torch.save([t.cpu() for t in out], sys.argv[1])
"""


def test_the_bounds_checked_build_gives_the_same(tmp_path):
    from rankmixer_feature_interaction_gb300 import build
    build.build(debug_bounds=True)
    got = []
    for variant in ("debug", "normal"):
        env = {k: v for k, v in os.environ.items() if not k.startswith("RM_")}
        env["PYTHONPATH"] = ROOT
        if variant == "debug":
            env["RM_LIBRARY"] = "debug"
        path = str(tmp_path / variant)
        r = subprocess.run([sys.executable, "-c", CHILD, path, variant], env=env, cwd=ROOT, capture_output=True, text=True,
                           timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        got.append(torch.load(path))
    assert len(got[0]) == len(got[1]) > 60
    for a, b in zip(*got):
        assert torch.equal(a, b)
