"""Refusals of the 8-bit operators at the ends of their ranges, on the host before anything is launched (no GPU
needed)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300 import build as rm_build
from rankmixer_feature_interaction_gb300.api import Fp8PFFN, Fp8Tensor

BAD, NO = _lib.RM_ERR_INVALID_ARG, _lib.RM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        rm_build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    yield (ctypes.addressof(buf) + 255) // 256 * 256
    del buf


def t8(p, cols, fmt=_lib.RM_E4M3):
    return _lib.rm_fp8_tensor(codes=p, scales=p + 4096, ld=(cols + 15) // 16 * 16,
                              lds=((cols + 127) // 128 + 3) // 4 * 4, format=fmt)


def test_sums_longer_than_the_accumulator_holds_are_refused(lib, mem):
    p, n = mem, ctypes.c_longlong()
    k = (1 << 19) + 16
    assert lib.rm_fp8_matmul(t8(p, k), t8(p, 32), None, p, 0, 1, 1, k, 32, 0, None) == NO
    assert "2^19" in _lib.rm_last_error()
    assert lib.rm_fp8_matmul(t8(p, k), t8(p, k), None, p, 0, 1, 1, k, 32, 1, None) == NO
    for D, F in ((k, 32), (32, k)):
        f = _lib.rm_fp8_pffn(t8(p, F), t8(p, D), p, p, 1, D, F)
        assert lib.rm_fp8_pffn_workspace(f, 1, _lib.RM_FP8_SERVE, ctypes.byref(n)) == NO
    b = (1 << 17) + 1
    assert lib.rm_fp8_wgrad(t8(p, 32), p, p, p, _lib.RM_BF16, b, 1, 32, 32, None) == NO
    assert "2^17" in _lib.rm_last_error()
    f = _lib.rm_fp8_pffn(t8(p, 32), t8(p, 32), p, p, 1, 32, 32)
    assert lib.rm_fp8_pffn_workspace(f, b, _lib.RM_FP8_BACKWARD, ctypes.byref(n)) == _lib.RM_OK
    kept = _lib.rm_fp8_kept(t8(p, 32), t8(p, 32), t8(p, 32))
    assert lib.rm_fp8_pffn_backward(f, p, 0, kept, p, 0, _lib.rm_fp8_grads(p, p, p, p, _lib.RM_BF16), b, p, n.value,
                                    None) == NO


def test_binding_refuses_sizes_that_do_not_fit_the_interface(lib, mem):
    """The C interface takes 32-bit sizes: 2^32 + 128 columns must not arrive there as 128."""
    p, n, q = mem, (1 << 32) + 128, t8(mem, 128)
    wide = t8(p, n)
    f = _lib.rm_fp8_pffn(t8(p, 32), t8(p, 32), p, p, 1, 32, 32)
    kept = _lib.rm_fp8_kept(t8(p, 32), t8(p, 32), t8(p, 32))
    calls = [lambda: _lib.rm_fp8_quantize(p, _lib.RM_F32, 1, n, n, wide, 0),
             lambda: _lib.rm_fp8_dequantize(wide, 1, n, p, _lib.RM_F32, n, 0),
             lambda: _lib.rm_fp8_quantize_weight(p, _lib.RM_F32, 1, n, 16, q, 0),
             lambda: _lib.rm_fp8_quantize_weight(p, _lib.RM_F32, 1, 16, n, wide, 0),
             lambda: _lib.rm_fp8_quantize_weight(p, _lib.RM_F32, (1 << 32) + 1, 16, 16, q, 0),
             lambda: _lib.rm_fp8_matmul(q, q, None, p, _lib.RM_F32, n, 1, 128, 128, False, 0),
             lambda: _lib.rm_fp8_matmul(q, wide, None, p, _lib.RM_F32, 1, 1, 128, n, False, 0),
             lambda: _lib.rm_fp8_matmul(wide, q, None, p, _lib.RM_F32, 1, 1, n, 128, False, 0),
             lambda: _lib.rm_fp8_wgrad(q, p, p, p, _lib.RM_F32, n, 1, 128, 128, 0),
             lambda: _lib.rm_fp8_pffn_workspace(f, n, _lib.RM_FP8_SERVE),
             lambda: _lib.rm_fp8_pffn_forward(f, p, 0, p, 0, None, n, p, 1 << 50, 0),
             lambda: _lib.rm_fp8_pffn_backward(f, p, 0, kept, p, 0, _lib.rm_fp8_grads(p, p, p, p, 0), n, p, 1 << 50, 0)]
    for i, call in enumerate(calls):
        with pytest.raises(_lib.RankMixerError) as e:
            call()
        assert e.value.status == BAD, i
    n, meta = (1 << 32) + 16, {"device": "meta"}
    w1 = Fp8Tensor(torch.empty((1, 16, n), dtype=torch.float8_e4m3fn, **meta),
                   torch.empty((1, 1, (n + 511) // 512 * 4), dtype=torch.uint8, **meta), n)
    w2 = Fp8Tensor(torch.empty((1, n, 16), dtype=torch.float8_e4m3fn, **meta),
                   torch.empty((1, (n + 127) // 128, 4), dtype=torch.uint8, **meta), 16)
    with pytest.raises(_lib.RankMixerError, match="32 bits"):
        Fp8PFFN(w1, torch.empty((1, n), **meta), w2, torch.empty((1, 16), **meta))


@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 128, (1 << 31) - 255])
def test_sizes_are_refused_before_they_overflow_when_rounded_up(lib, mem, n):
    """2^31 - 1 columns round up to -2^31 in 32 bits: the row of scales would pass as long enough at any length."""
    p, q = mem, t8(mem, 128)
    short = _lib.rm_fp8_tensor(p, p + 4096, (n + 15) // 16 * 16, 4, _lib.RM_E4M3)
    wide = t8(p, n)
    for t in (short, wide):
        assert lib.rm_fp8_quantize(p, _lib.RM_F32, 1, n, n, t, None) == BAD
        assert lib.rm_fp8_dequantize(t, 1, n, p, _lib.RM_F32, n, None) == BAD
        assert lib.rm_fp8_quantize_weight(p, _lib.RM_F32, 1, 16, n, t, None) == BAD
        assert lib.rm_fp8_matmul(q, t, None, p, _lib.RM_F32, 1, 1, 128, n, 0, None) == BAD
        assert lib.rm_fp8_matmul(t, q, None, p, _lib.RM_F32, 1, 1, n, 128, 0, None) in (BAD, NO)
        assert lib.rm_fp8_wgrad(t, p, p, p, _lib.RM_F32, 1, 1, n, 128, None) == BAD
    assert lib.rm_fp8_matmul(q, q, None, p, _lib.RM_F32, n, 1, 128, 128, 0, None) == BAD
    assert lib.rm_fp8_matmul(q, q, None, p, _lib.RM_F32, 1, 1, 128, n, 1, None) == BAD
    assert lib.rm_fp8_wgrad(q, p, p, p, _lib.RM_F32, 1, 1, 128, n // 8 * 8, None) == BAD


def test_the_package_imports_on_a_torch_without_cuda():
    """A torch built without CUDA has none of torch._C's stream and device functions."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from rankmixer_feature_interaction_gb300 import api\n"
            "try:\n    api.fp8_quantize(torch.zeros(2, 3))\n"
            "except ValueError as e:\n    assert 'CUDA' in str(e), e\n"
            "else:\n    raise SystemExit('not refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env={**os.environ, "PYTHONPATH": root},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
