"""The 8-bit operators' refusals, checked on the host before anything is launched (no GPU needed),
the binding's structures against the header, and the tests' own restatement of the format."""
import ctypes
import os
import re

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300 import build as rm_build
from rankmixer_feature_interaction_gb300.api import Fp8PFFN, Fp8Tensor, fp8_matmul, fp8_quantize
from tests import fp8_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rankmixer.h")
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


def t8(p, cols, fmt=_lib.RM_E4M3, **kw):
    f = dict(codes=p, scales=p + 4096, ld=(cols + 15) // 16 * 16, lds=((cols + 127) // 128 + 3) // 4 * 4, format=fmt)
    f.update(kw)
    return _lib.rm_fp8_tensor(**f)


BAD_TENSORS = [("codes", 0), ("scales", 0), ("codes", 8), ("scales", 2), ("ld", 192), ("ld", 201), ("lds", 0),
               ("lds", 2), ("lds", 3), ("format", 2)]


def bad_tensor(p, field, v, cols=200):
    """A tensor of 200 columns with one field wrong: codes / scales by an offset from an aligned address (0: NULL)."""
    if field in ("codes", "scales"):
        v = p + v if v else None
    return t8(p, cols, **{field: v})


@pytest.mark.parametrize("field,v", BAD_TENSORS)
def test_every_call_refuses_a_bad_tensor(lib, mem, field, v):
    bad, good = bad_tensor(mem, field, v), t8(mem, 200)
    p = mem
    assert lib.rm_fp8_quantize(p, _lib.RM_F32, 3, 200, 200, bad, None) == BAD
    assert lib.rm_fp8_quantize_weight(p, _lib.RM_F32, 2, 3, 200, bad, None) == BAD
    assert lib.rm_fp8_dequantize(bad, 3, 200, p, _lib.RM_F32, 200, None) == BAD
    assert lib.rm_fp8_matmul(bad, good, None, p, _lib.RM_F32, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_matmul(good, bad, None, p, _lib.RM_F32, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_wgrad(bad, p, p, p, _lib.RM_F32, 3, 2, 200, 200, None) == BAD
    n = ctypes.c_longlong()
    f = _lib.rm_fp8_pffn(bad_tensor(p, field, v, 208) if field != "ld" else t8(p, 208, ld=200), t8(p, 208), p, p, 2,
                         208, 208)
    assert lib.rm_fp8_pffn_workspace(f, 3, 0, ctypes.byref(n)) == BAD
    assert lib.rm_fp8_pffn_forward(f, p, 0, p, 0, None, 3, p, 1 << 30, None) == BAD


def test_quantize_refusals(lib, mem):
    p, q = mem, t8(mem, 200)
    ok = dict(X=p, dtype=_lib.RM_F32, rows=3, cols=200, ldx=200, out=q)

    def call(**kw):
        a = {**ok, **kw}
        return lib.rm_fp8_quantize(a["X"], a["dtype"], a["rows"], a["cols"], a["ldx"], a["out"], None)
    for kw in (dict(X=None), dict(dtype=2), dict(rows=0), dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(ldx=199),
               dict(X=p + 2), dict(out=None)):
        assert call(**kw) == BAD, kw
    assert call(dtype=_lib.RM_BF16, X=p + 1) == BAD
    assert lib.rm_fp8_dequantize(q, 3, 200, None, 0, 200, None) == BAD
    assert lib.rm_fp8_dequantize(q, 3, 200, p, 0, 199, None) == BAD
    assert lib.rm_fp8_dequantize(q, 0, 200, p, 0, 200, None) == BAD
    assert lib.rm_fp8_dequantize(q, 3, 200, p, 3, 200, None) == BAD
    assert lib.rm_fp8_dequantize(None, 3, 200, p, 0, 200, None) == BAD
    assert lib.rm_fp8_dequantize(q, 3, 200, p + 2, 0, 200, None) == BAD
    assert lib.rm_fp8_quantize_weight(None, 0, 2, 3, 200, q, None) == BAD
    assert lib.rm_fp8_quantize_weight(p, 5, 2, 3, 200, q, None) == BAD
    assert lib.rm_fp8_quantize_weight(p, 0, 0, 3, 200, q, None) == BAD
    assert lib.rm_fp8_quantize_weight(p, 0, 2, 3, 200, t8(p, 200, _lib.RM_E5M2), None) == NO
    assert "e4m3" in _lib.rm_last_error()


def test_matmul_and_wgrad_refusals(lib, mem):
    p, q = mem, t8(mem, 200)
    for B, T, K, N in ((0, 2, 200, 200), (3, 0, 200, 200), (3, 2, 0, 200), (3, 2, 200, 0), (-1, 2, 200, 200),
                       (3, 65536, 200, 200), (65536, 32768, 200, 200)):
        assert lib.rm_fp8_matmul(q, q, None, p, 0, B, T, K, N, 0, None) == BAD
        assert lib.rm_fp8_wgrad(q, p, p, p, 0, B, T, K, N, None) == BAD
    assert lib.rm_fp8_matmul(q, q, None, None, 0, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_matmul(q, q, None, p + 4, 0, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_matmul(q, q, p + 4, p, 0, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_matmul(q, q, None, p, 2, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_matmul(None, q, None, p, 0, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_matmul(q, None, None, p, 0, 3, 2, 200, 200, 0, None) == BAD
    assert lib.rm_fp8_matmul(q, t8(p, 200, _lib.RM_E5M2), None, p, 0, 3, 2, 200, 200, 0, None) == NO
    # the weight's row length is N, or K when it is read transposed
    assert lib.rm_fp8_matmul(q, q, None, p, 0, 3, 2, 200, 300, 0, None) == BAD
    assert lib.rm_fp8_matmul(t8(p, 300), q, None, p, 0, 3, 2, 300, 200, 1, None) == BAD
    assert lib.rm_fp8_wgrad(q, None, p, p, 0, 3, 2, 200, 200, None) == BAD
    assert lib.rm_fp8_wgrad(q, p, None, None, 0, 3, 2, 200, 200, None) == BAD
    assert lib.rm_fp8_wgrad(q, p, p, p, 7, 3, 2, 200, 200, None) == BAD
    assert lib.rm_fp8_wgrad(q, p + 2, p, p, 0, 3, 2, 200, 200, None) == BAD
    assert lib.rm_fp8_wgrad(q, p, p, p, 0, 3, 2, 200, 204, None) == NO
    assert lib.rm_fp8_wgrad(t8(p, 200, _lib.RM_E5M2), p, p, p, 0, 3, 2, 200, 200, None) == NO
    # lengths summed over
    big = (1 << 27) + 16
    assert lib.rm_fp8_matmul(t8(p, big), t8(p, 200), None, p, 0, 1, 1, big, 200, 0, None) == NO
    assert lib.rm_fp8_wgrad(q, p, p, p, 0, big, 1, 200, 200, None) == NO
    assert "2^27" in _lib.rm_last_error()


def test_pffn_refusals(lib, mem):
    p, n = mem, ctypes.c_longlong(7)
    f = _lib.rm_fp8_pffn(t8(p, 416), t8(p, 208), p, p, 2, 208, 416)
    assert lib.rm_fp8_pffn_workspace(f, 5, _lib.RM_FP8_SERVE, ctypes.byref(n)) == _lib.RM_OK
    serve = n.value
    assert serve >= 5 * 2 * (208 + 416)                       # at least the two 8-bit operands
    assert lib.rm_fp8_pffn_workspace(f, 5, 3, ctypes.byref(n)) == BAD and n.value == 0
    assert lib.rm_fp8_pffn_workspace(f, 0, 0, ctypes.byref(n)) == BAD
    assert lib.rm_fp8_pffn_workspace(None, 5, 0, ctypes.byref(n)) == BAD
    assert lib.rm_fp8_pffn_workspace(f, 5, 0, None) == BAD
    for D, F in ((200, 416), (208, 408)):
        g = _lib.rm_fp8_pffn(t8(p, 416), t8(p, 208), p, p, 2, D, F)
        assert lib.rm_fp8_pffn_workspace(g, 5, 0, ctypes.byref(n)) == NO
    for b1, b2 in ((None, p), (p, None), (p + 4, p)):
        g = _lib.rm_fp8_pffn(t8(p, 416), t8(p, 208), b1, b2, 2, 208, 416)
        assert lib.rm_fp8_pffn_workspace(g, 5, 0, ctypes.byref(n)) == BAD
    fwd = lib.rm_fp8_pffn_forward
    assert fwd(f, p, 0, p, 0, None, 5, p, serve - 1, None) == BAD and "work_bytes" in _lib.rm_last_error()
    assert fwd(f, p, 0, p, 0, None, 5, None, serve, None) == BAD
    assert fwd(f, p, 0, p, 0, None, 5, p + 8, serve, None) == BAD
    assert fwd(f, None, 0, p, 0, None, 5, p, serve, None) == BAD
    assert fwd(f, p, 0, None, 0, None, 5, p, serve, None) == BAD
    assert fwd(f, p, 3, p, 0, None, 5, p, serve, None) == BAD
    assert fwd(f, p + 2, 1, p, 0, None, 5, p, serve, None) == BAD
    kept = _lib.rm_fp8_kept(t8(p, 208), t8(p, 416, _lib.RM_E5M2), t8(p, 416))
    assert fwd(f, p, 0, p, 0, kept, 5, p, 1 << 40, None) == NO
    bwd = lib.rm_fp8_pffn_backward
    kept = _lib.rm_fp8_kept(t8(p, 208), t8(p, 416), t8(p, 416))
    g = _lib.rm_fp8_grads(p, p, p, p, 0)
    assert lib.rm_fp8_pffn_workspace(f, 5, _lib.RM_FP8_BACKWARD, ctypes.byref(n)) == _lib.RM_OK
    assert bwd(f, p, 0, kept, p, 0, g, 5, p, n.value - 1, None) == BAD
    assert bwd(f, None, 0, kept, p, 0, g, 5, p, n.value, None) == BAD
    assert bwd(f, p, 0, None, p, 0, g, 5, p, n.value, None) == BAD
    assert bwd(f, p, 0, kept, p, 0, None, 5, p, n.value, None) == BAD
    assert bwd(f, p, 0, kept, p, 0, _lib.rm_fp8_grads(p, None, p, p, 0), 5, p, n.value, None) == BAD
    assert bwd(f, p, 0, kept, p, 0, _lib.rm_fp8_grads(p, p + 4, p, p, 0), 5, p, n.value, None) == BAD
    assert bwd(f, p, 0, kept, p, 0, _lib.rm_fp8_grads(p, p, p, p, 5), 5, p, n.value, None) == BAD
    assert bwd(f, p, 0, kept, p, 9, g, 5, p, n.value, None) == BAD
    assert bwd(f, p, 0, _lib.rm_fp8_kept(t8(p, 208), t8(p, 208), t8(p, 416)), p, 0, g, 5, p, n.value, None) == BAD


def test_binding_refuses_tensors_that_are_not_of_the_format():
    codes, scales = torch.zeros((3, 2, 208), dtype=torch.float8_e4m3fn), torch.zeros((3, 2, 4), dtype=torch.uint8)
    assert Fp8Tensor(codes, scales, 200).shape == (3, 2, 200)
    for c, s, n in ((codes.view(torch.uint8), scales, 200), (codes, scales.view(torch.int8), 200), (codes, scales, 209),
                    (codes, scales, 0), (codes, scales[0], 200), (torch.zeros((3, 2, 528)).to(codes.dtype), scales, 520),
                    (codes.transpose(0, 1), scales.transpose(0, 1), 200)):
        with pytest.raises(ValueError):
            Fp8Tensor(c, s, n)
    w = Fp8Tensor(torch.zeros((2, 208, 208)).to(codes.dtype), torch.zeros((2, 2, 4), dtype=torch.uint8), 208)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):      # no CUDA tensors
        fp8_matmul(Fp8Tensor(codes, scales, 200), w)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        fp8_quantize(torch.zeros(3, 2))
    with pytest.raises(ValueError):                                      # W2 is not [T, F, D]
        Fp8PFFN(w, torch.zeros(2, 208), Fp8Tensor(torch.zeros((2, 16, 208)).to(codes.dtype),
                                                  torch.zeros((2, 1, 4), dtype=torch.uint8), 208), torch.zeros(2, 208))


def test_structures_match_the_header():
    text = open(HEADER, encoding="utf-8").read()
    for name, struct in (("rm_fp8_tensor", _lib.rm_fp8_tensor), ("rm_fp8_pffn", _lib.rm_fp8_pffn),
                         ("rm_fp8_kept", _lib.rm_fp8_kept), ("rm_fp8_grads", _lib.rm_fp8_grads)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [re.sub(r".*[\s*]", "", f.strip()) for d in body.split(";") if d.strip() for f in d.split(",")]
        assert fields == [f for f, _ in struct._fields_], name


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_the_reference_format_on_values_with_known_answers(fmt):
    big = 0.875 * 2.0 ** ref.TOP[fmt]
    x = torch.zeros((6, 256))
    x[0, 3] = big                                    # exactly the largest: scale 1
    x[1, 3], x[1, 130] = big * (1 + 2.0 ** -20), -big * 4   # just above: scale 2; another block of its own
    x[2, 0], x[2, 1] = float("inf"), 1.0             # does not count
    x[3, 0], x[3, 1] = float("nan"), -big / 2
    x[4, 0] = 2.0 ** -149                            # the smallest float: E = 1
    codes, E = ref.quantise(x, fmt)
    assert E.tolist() == [[127, 127], [128, 129], [127 - ref.TOP[fmt] + 1, 127], [126, 127], [1, 127], [127, 127]]
    v = codes.view(ref.F8[fmt]).double()
    assert v[0, 3] == big and v[1, 3] == big / 2 and v[1, 130] == -big and v[2, 0].isnan() and v[3, 0].isnan()
    assert v[2, 1] == 2.0 ** (ref.TOP[fmt] - 1) and v[3, 1] == -big and v[4, 0] == 0 and not v[5].any()
