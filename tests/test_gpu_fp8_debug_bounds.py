"""The 8-bit operators in the bounds-checked build: no launcher check fails on valid calls, and every result is the
normal build's, bit for bit."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = r"""
import sys, torch
from rankmixer_feature_interaction_gb300 import _lib, api
_lib.load()
maps = open("/proc/self/maps").read()
assert ("librankmixer_debug.so" in maps) == (sys.argv[2] == "debug")
out, g = [], torch.Generator(device="cuda").manual_seed(5)
def rnd(*s): return torch.randn(s, generator=g, device="cuda")
# streamed weights (one tile's K shared too), pairs of thread blocks, odd sizes, both directions and formats
for B, T, K, N in ((1, 8, 2048, 512), (40, 3, 200, 130), (300, 20, 272, 520), (257, 2, 1001, 333)):
    X = rnd(B, T, K)
    for fmt in ("e4m3", "e5m2"):
        q = api.fp8_quantize(X, fmt)
        out += [q.codes.view(torch.uint8)[..., :K], q.scales[..., :(K + 127) // 128], api.fp8_dequantize(q),
                api.fp8_dequantize(q, "f32")]
        for w, trans in ((api.fp8_quantize_weight(rnd(T, K, N)), False), (api.fp8_quantize_weight(rnd(T, N, K)), True)):
            out += [api.fp8_matmul(q, w, rnd(T, N), "f32", trans), api.fp8_matmul(q, w, None, "bf16", trans)]
    out += api.fp8_wgrad(api.fp8_quantize(X[..., 1:]), rnd(B, T, 8 * (N // 8)).to(torch.bfloat16))
for B, T, D, F in ((3, 4, 128, 256), (70, 2, 144, 400), (300, 20, 144, 400)):
    m = api.Fp8PFFN(rnd(T, D, F), rnd(T, F), rnd(T, F, D), rnd(T, D))
    X = rnd(B, T, D)
    V, kept = m.forward_train(X, "f32")
    for dV, grad in ((X, "f32"), (X.to(torch.bfloat16), "bf16")):
        dX, grads = m.backward(dV, kept, grad_dtype=grad)
        out += [dX, *grads.values()]
    out += [V, m.forward(X)]
assert api.fp8_sync_status() == _lib.RM_OK
torch.save([t.cpu() for t in out], sys.argv[1])
"""


def test_bounds_checked_8bit_operators_match_the_normal_build(tmp_path):
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
    assert len(got[0]) == len(got[1]) > 80
    for a, b in zip(*got):
        assert torch.equal(a, b)
