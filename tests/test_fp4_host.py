"""Refusals of the 4-bit operators and of the experts' rows, checked on the host before anything is launched (no GPU
needed), the binding's structures against the header, and the tests' own restatements."""
import ctypes
import os
import re

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300 import build as rm_build
from rankmixer_feature_interaction_gb300.api import (Fp4MoE, Fp4PFFN, Fp4Tensor, expert_sort, fp4_dequantize, fp4_matmul,
                                                     fp4_quantize, fp4_quantize_weight)
from tests import fp4_reference as ref
from tests.test_nvtx_ranges import ranges

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rankmixer.h")
BAD, NO, OK = _lib.RM_ERR_INVALID_ARG, _lib.RM_ERR_UNSUPPORTED, _lib.RM_OK
MAX = 0x7fffffff - 511


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


def act(p, cols, **kw):
    f = dict(codes=p, scales=p + 4096, ld=16 * ((cols + 31) // 32), lds=((cols + 31) // 32 + 15) // 16 * 16)
    f.update(kw)
    return _lib.rm_fp4_tensor(**f)


def wt(p, K, **kw):
    f = dict(codes=p, scales=p + 4096, ld=16 * ((K + 31) // 32), lds=2 * ((K + 255) // 256))
    f.update(kw)
    return _lib.rm_fp4_tensor(**f)


def rows(p, B=5, T=2, E=3, **kw):
    f = dict(offsets=p, source=p + 256, slot=p + 512, tiles=p + 1024, B=B, T=T, E=E)
    f.update(kw)
    return _lib.rm_expert_rows(**f)


@pytest.mark.parametrize("field,v", [("codes", None), ("scales", None), ("codes", 8), ("scales", 8), ("ld", 96), ("ld", 120),
                                     ("lds", 6), ("lds", 0), ("lds", 24)])
def test_every_call_refuses_bad_activations(lib, mem, field, v):
    """Of 200 columns: 7 blocks, 112 bytes of codes, 16 of scales."""
    p = mem
    bad = act(p, 200, **{field: p + v if field in ("codes", "scales") and v else v})
    w, r = wt(p, 200), rows(p)
    assert lib.rm_fp4_quantize(p, 0, 3, 200, 200, bad, None) == BAD
    assert lib.rm_fp4_dequantize(bad, 3, 200, p, 0, 200, None) == BAD
    assert lib.rm_fp4_matmul(bad, w, None, p, 0, 3, 2, 200, 200, None) == BAD
    assert lib.rm_fp4_expert_gather(p, 0, r, bad, 7, 200, None) == BAD
    assert lib.rm_fp4_expert_matmul(bad, w, r, None, p, 0, 7, 200, 200, None) == BAD


@pytest.mark.parametrize("field,v", [("codes", None), ("scales", None), ("codes", 8), ("scales", 4), ("ld", 96), ("ld", 120),
                                     ("lds", 1), ("lds", 3), ("lds", 4)])
def test_every_call_refuses_bad_weights(lib, mem, field, v):
    p, n = mem, ctypes.c_longlong()
    kw = {field: p + v if field in ("codes", "scales") and v else v}
    bad, x, r = wt(p, 200, **kw), act(p, 200), rows(p)
    assert lib.rm_fp4_quantize_weight(p, 0, 2, 200, 30, bad, None) == BAD
    assert lib.rm_fp4_matmul(x, bad, None, p, 0, 3, 2, 200, 200, None) == BAD
    assert lib.rm_fp4_expert_matmul(x, bad, r, None, p, 0, 7, 200, 200, None) == BAD
    bad = wt(p, 224, **kw)                               # 7 blocks too, and a multiple of 32
    for w1, w2 in ((bad, wt(p, 224)), (wt(p, 224), bad)):
        f = _lib.rm_fp4_pffn(w1, w2, p, p, 2, 224, 224)
        assert lib.rm_fp4_pffn_workspace(f, 3, ctypes.byref(n)) == BAD and n.value == 0
        assert lib.rm_fp4_pffn_forward(f, p, 0, p, 0, 3, p, 1 << 40, None) == BAD
        m = _lib.rm_fp4_moe(w1, w2, p, p, 2, 3, 224, 224)
        assert lib.rm_fp4_moe_workspace(m, 3, ctypes.byref(n)) == BAD and n.value == 0
        assert lib.rm_fp4_moe_forward(m, p, 0, p, p, 0, 3, p, 1 << 40, None) == BAD


def test_quantize_refusals(lib, mem):
    p, q = mem, act(mem, 200)
    ok = dict(X=p, dtype=_lib.RM_F32, rows=3, cols=200, ldx=200, out=q)

    def call(**kw):
        a = {**ok, **kw}
        return lib.rm_fp4_quantize(a["X"], a["dtype"], a["rows"], a["cols"], a["ldx"], a["out"], None)
    for kw in (dict(X=None), dict(dtype=2), dict(rows=0), dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=-5),
               dict(cols=MAX + 1), dict(ldx=199), dict(X=p + 2), dict(out=None), dict(dtype=_lib.RM_BF16, X=p + 1)):
        assert call(**kw) == BAD, kw
    assert lib.rm_fp4_dequantize(q, 3, 200, None, 0, 200, None) == BAD
    assert lib.rm_fp4_dequantize(q, 3, 200, p, 0, 199, None) == BAD
    assert lib.rm_fp4_dequantize(q, 3, 200, p + 2, 0, 200, None) == BAD
    assert lib.rm_fp4_dequantize(q, 3, 200, p, 4, 200, None) == BAD
    assert lib.rm_fp4_dequantize(None, 3, 200, p, 0, 200, None) == BAD
    w, qw = wt(p, 200), lib.rm_fp4_quantize_weight
    for a in ((None, 0, 2, 200, 30, w), (p, 5, 2, 200, 30, w), (p, 0, 0, 200, 30, w), (p, 0, 2, 0, 30, w),
              (p, 0, 2, 200, 0, w), (p, 0, 65536, 200, 30, w), (p + 2, 0, 2, 200, 30, w), (p, 0, 2, 200, 30, None),
              (p, 0, 2, 200, MAX + 1, w)):
        assert qw(*a, None) == BAD, a
    big = (1 << 19) + 1
    assert qw(p, 0, 2, big, 30, wt(p, big), None) == NO


def test_matmul_refusals(lib, mem):
    p = mem
    x, w = act(p, 200), wt(p, 200)
    mm = lib.rm_fp4_matmul
    for B, T, K, N in ((0, 2, 200, 30), (3, 0, 200, 30), (3, 2, 0, 30), (3, 2, 200, 0), (-1, 2, 200, 30), (3, 65536, 200, 30),
                       (3, 2, 200, MAX + 1), (MAX + 1, 1, 200, 30), (1 << 30, 2, 200, 30)):
        assert mm(x, w, None, p, 0, B, T, K, N, None) == BAD, (B, T, K, N)
    assert mm(x, w, None, None, 0, 3, 2, 200, 30, None) == BAD
    assert mm(x, w, None, p + 8, 0, 3, 2, 200, 30, None) == BAD
    assert mm(x, w, p + 4, p, 0, 3, 2, 200, 30, None) == BAD
    assert mm(x, w, None, p, 2, 3, 2, 200, 30, None) == BAD
    assert mm(None, w, None, p, 0, 3, 2, 200, 30, None) == BAD
    assert mm(x, None, None, p, 0, 3, 2, 200, 30, None) == BAD
    big = (1 << 19) + 1
    assert mm(act(p, big), wt(p, big), None, p, 0, 3, 2, big, 30, None) == NO and "2^19" in _lib.rm_last_error()


def test_ffn_refusals(lib, mem):
    p, n = mem, ctypes.c_longlong(7)
    f = _lib.rm_fp4_pffn(wt(p, 224), wt(p, 416), p, p, 2, 224, 416)
    assert lib.rm_fp4_pffn_workspace(f, 5, ctypes.byref(n)) == OK
    need = n.value
    assert need >= 5 * 2 * (224 + 416) // 2
    for B in (0, -1, MAX + 1, 1 << 30):
        assert lib.rm_fp4_pffn_workspace(f, B, ctypes.byref(n)) == BAD and n.value == 0
    assert lib.rm_fp4_pffn_workspace(None, 5, ctypes.byref(n)) == BAD
    assert lib.rm_fp4_pffn_workspace(f, 5, None) == BAD
    for D, F in ((200, 416), (224, 400)):
        g = _lib.rm_fp4_pffn(wt(p, D), wt(p, F), p, p, 2, D, F)
        assert lib.rm_fp4_pffn_workspace(g, 5, ctypes.byref(n)) == NO
    for b1, b2 in ((None, p), (p, None), (p + 4, p)):
        g = _lib.rm_fp4_pffn(wt(p, 224), wt(p, 416), b1, b2, 2, 224, 416)
        assert lib.rm_fp4_pffn_workspace(g, 5, ctypes.byref(n)) == BAD
    fwd = lib.rm_fp4_pffn_forward
    assert fwd(f, p, 0, p, 0, 5, p, need - 1, None) == BAD and "work_bytes" in _lib.rm_last_error()
    for a in ((None, 0, p, 0, 5, p), (p, 0, None, 0, 5, p), (p, 3, p, 0, 5, p), (p, 0, p, 3, 5, p), (p + 8, 0, p, 0, 5, p),
              (p, 0, p + 8, 0, 5, p), (p, 0, p, 0, 5, None), (p, 0, p, 0, 5, p + 8), (p, 0, p, 0, 0, p)):
        assert fwd(f, *a, need, None) == BAD, a
    m = _lib.rm_fp4_moe(wt(p, 224), wt(p, 416), p, p, 2, 3, 224, 416)
    assert lib.rm_fp4_moe_workspace(m, 5, ctypes.byref(n)) == OK
    need = n.value
    assert need >= 5 * 6 * ((224 + 416) // 2 + 2 * 224)
    for T, E, B in ((0, 3, 5), (2, 0, 5), (2, 3, 0), (300, 300, 5), (2, 3, 1 << 29)):
        g = _lib.rm_fp4_moe(wt(p, 224), wt(p, 416), p, p, T, E, 224, 416)
        assert lib.rm_fp4_moe_workspace(g, B, ctypes.byref(n)) == BAD and n.value == 0
    fwd = lib.rm_fp4_moe_forward
    assert fwd(m, p, 0, p, p, 0, 5, p, need - 1, None) == BAD and "work_bytes" in _lib.rm_last_error()
    for a in ((None, 0, p, p, 0, 5, p), (p, 0, None, p, 0, 5, p), (p, 0, p, None, 0, 5, p), (p, 2, p, p, 0, 5, p),
              (p, 0, p, p, 2, 5, p), (p + 8, 0, p, p, 0, 5, p), (p, 0, p + 2, p, 0, 5, p), (p, 0, p, p + 8, 0, 5, p),
              (p, 0, p, p, 0, 5, None)):
        assert fwd(m, *a, need, None) == BAD, a


def test_rows_refusals(lib, mem):
    p, n = mem, ctypes.c_longlong()
    r = rows(p)
    for B, T, E in ((0, 2, 3), (5, 0, 3), (5, 2, 0), (-1, 2, 3), (5, 256, 256), (1 << 30, 2, 1), (MAX + 1, 1, 1)):
        assert lib.rm_expert_sort_workspace(B, T, E, ctypes.byref(n)) == BAD and n.value == 0
        assert lib.rm_expert_sort(p, rows(p, B, T, E), p, 1 << 40, None) == BAD
        assert lib.rm_expert_gather(p, 0, rows(p, B, T, E), p, 7, 8, None) == BAD
    assert lib.rm_expert_sort_workspace(5, 2, 3, None) == BAD
    for kw in (dict(offsets=None), dict(source=None), dict(slot=None), dict(tiles=None), dict(tiles=p + 4), dict(slot=p + 2)):
        bad = rows(p, **kw)
        assert lib.rm_expert_sort(p, bad, p, 1 << 40, None) == BAD
        assert lib.rm_expert_gather(p, 0, bad, p, 7, 8, None) == BAD
        assert lib.rm_fp4_expert_gather(p, 0, bad, act(p, 8), 7, 8, None) == BAD
        assert lib.rm_expert_combine(p, 0, bad, p, p, 0, 7, 8, None) == BAD
        assert lib.rm_expert_combine_backward(p, p, 0, bad, p, p, p, 7, 8, None) == BAD
        assert lib.rm_fp4_expert_matmul(act(p, 8), wt(p, 8), bad, None, p, 0, 7, 8, 8, None) == BAD
    assert lib.rm_expert_sort(None, r, p, 1 << 40, None) == BAD
    assert lib.rm_expert_sort(p + 2, r, p, 1 << 40, None) == BAD
    many = rows(p, 100, 2, 3)
    assert lib.rm_expert_sort_workspace(100, 2, 3, ctypes.byref(n)) == OK and n.value > 0
    assert lib.rm_expert_sort(p, many, p, n.value - 1, None) == BAD
    assert lib.rm_expert_sort(p, many, None, n.value, None) == BAD
    for c in (lambda X, dt, Xs, k, D: lib.rm_expert_gather(X, dt, r, Xs, k, D, None),
              lambda X, dt, Xs, k, D: lib.rm_expert_combine(Xs, dt, r, None, X, dt, k, D, None),
              lambda X, dt, Xs, k, D: lib.rm_expert_combine_backward(X, Xs, dt, r, p, p, p, k, D, None)):
        for a in ((None, 0, p, 7, 8), (p, 0, None, 7, 8), (p, 3, p, 7, 8), (p, 0, p, -1, 8), (p, 0, p, 1 << 31, 8),
                  (p, 0, p, 7, 0), (p, 0, p, 7, MAX + 1), (p + 2, 0, p, 7, 8), (p, 0, p + 2, 7, 8), (p + 1, 1, p, 7, 8)):
            assert c(*a) == BAD, a
    assert lib.rm_expert_combine(p, 0, r, p + 2, p, 0, 7, 8, None) == BAD
    for G, dY, dG in ((None, p, p), (p, None, p), (p, p, None), (p + 2, p, p), (p, p, p + 2), (p, p + 2, p)):
        assert lib.rm_expert_combine_backward(p, p, 0, r, G, dY, dG, 7, 8, None) == BAD
    # no rows: nothing to launch, whatever the buffers
    assert lib.rm_expert_gather(p, 0, r, None, 0, 8, None) == OK
    assert lib.rm_fp4_expert_gather(p, 0, r, None, 0, 8, None) == OK
    assert lib.rm_fp4_expert_matmul(None, wt(p, 8), r, None, None, 0, 0, 8, 8, None) == OK
    mm = lib.rm_fp4_expert_matmul
    assert mm(act(p, 8), wt(p, 8), r, None, None, 0, 7, 8, 8, None) == BAD
    assert mm(act(p, 8), wt(p, 8), r, p + 4, p, 0, 7, 8, 8, None) == BAD
    assert mm(act(p, 8), wt(p, 8), r, None, p, 2, 7, 8, 8, None) == BAD
    assert mm(act(p, 8), wt(p, 8), r, None, p, 0, 7, 0, 8, None) == BAD


def test_the_binding_refuses_sizes_past_32_bits():
    q = _lib.rm_fp4_tensor()
    r = _lib.rm_expert_rows()
    for call in (lambda: _lib.rm_fp4_quantize(0, 0, 1, 1 << 32, 1 << 32, q, 0),
                 lambda: _lib.rm_fp4_quantize_weight(0, 0, 1, (1 << 32) + 1, 1, q, 0),
                 lambda: _lib.rm_fp4_dequantize(q, 1, 1 << 32, 0, 0, 1 << 32, 0),
                 lambda: _lib.rm_fp4_matmul(q, q, None, 0, 0, (1 << 32) + 1, 1, 1, 1, 0),
                 lambda: _lib.rm_fp4_pffn_workspace(_lib.rm_fp4_pffn(), (1 << 32) + 1),
                 lambda: _lib.rm_fp4_moe_workspace(_lib.rm_fp4_moe(), (1 << 32) + 1),
                 lambda: _lib.rm_expert_sort_workspace((1 << 32) + 1, 1, 1),
                 lambda: _lib.rm_expert_gather(0, 0, r, 0, 1, (1 << 32) + 1, 0),
                 lambda: _lib.rm_fp4_expert_gather(0, 0, r, q, 1, (1 << 32) + 1, 0),
                 lambda: _lib.rm_expert_combine(0, 0, r, None, 0, 0, 1, (1 << 32) + 1, 0),
                 lambda: _lib.rm_expert_combine_backward(0, 0, 0, r, 0, 0, 0, 1, (1 << 32) + 1, 0),
                 lambda: _lib.rm_fp4_expert_matmul(q, q, r, None, 0, 0, 1, (1 << 32) + 1, 1, 0)):
        with pytest.raises(_lib.RankMixerError, match="32 bits"):
            call()


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_binding_refuses_tensors_that_are_not_of_the_format():
    assert Fp4Tensor(u8(3, 2, 112), u8(3, 2, 16), 200).shape == (3, 2, 200)
    assert Fp4Tensor(u8(2, 130, 112), u8(2, 2, 2, 512), 200, weight=True).shape == (2, 200, 130)
    for c, s, n, w in ((u8(3, 2, 112).view(torch.int8), u8(3, 2, 16), 200, False), (u8(3, 2, 96), u8(3, 2, 16), 200, False),
                       (u8(3, 2, 112), u8(3, 2, 6), 200, False), (u8(3, 2, 112), u8(2, 2, 16), 200, False),
                       (u8(3, 2, 112), u8(3, 2, 16), 0, False),
                       (u8(3, 2, 112).transpose(0, 1), u8(3, 2, 16).transpose(0, 1), 200, False),
                       (u8(2, 130, 112), u8(2, 1, 2, 512), 200, True), (u8(2, 130, 112), u8(2, 2, 1, 512), 200, True),
                       (u8(2, 130, 112), u8(2, 2, 2, 256), 200, True), (u8(112), u8(1, 2, 512), 200, True)):
        with pytest.raises(ValueError):
            Fp4Tensor(c, s, n, w)
    x, w = Fp4Tensor(u8(3, 2, 112), u8(3, 2, 16), 200), Fp4Tensor(u8(2, 224, 112), u8(2, 2, 2, 512), 224, weight=True)
    for call in (lambda: fp4_matmul(x, w), lambda: fp4_matmul(w, x), lambda: fp4_quantize(torch.zeros(3, 2)),
                 lambda: fp4_quantize_weight(torch.zeros(3, 2, 2)), lambda: fp4_dequantize(x),
                 lambda: expert_sort(torch.zeros(3, 2, 2)), lambda: Fp4PFFN(w, torch.zeros(2, 224), x, torch.zeros(2, 224)),
                 lambda: Fp4MoE(w, torch.zeros(2, 224), w, torch.zeros(2, 224)),
                 lambda: Fp4PFFN(w, torch.zeros(2, 224), w, torch.zeros(2, 225))):
        with pytest.raises((ValueError, AssertionError, RuntimeError)):          # no CUDA tensors, or that do not fit
            call()


def test_structures_match_the_header():
    text = open(HEADER, encoding="utf-8").read()
    for struct in (_lib.rm_fp4_tensor, _lib.rm_fp4_pffn, _lib.rm_expert_rows, _lib.rm_fp4_moe):
        name = struct.__name__
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [re.sub(r".*[\s*]", "", f.strip()) for d in body.split(";") if d.strip() for f in d.split(",")]
        assert fields == [f for f, _ in struct._fields_], name


def test_launches_are_ranged(tmp_path):
    """Without a device: the launch fails, in its range."""
    got = ranges(tmp_path, """
        import ctypes
        from rankmixer_feature_interaction_gb300 import _lib
        buf = ctypes.create_string_buffer(1 << 16)
        p = (ctypes.addressof(buf) + 255) // 256 * 256
        q, w = _lib.rm_fp4_tensor(p, p + 4096, 112, 16), _lib.rm_fp4_tensor(p, p + 4096, 112, 2)
        r = _lib.rm_expert_rows(p, p, p, p, 5, 2, 3)
        for call in (lambda: _lib.rm_fp4_quantize(p, 0, 3, 200, 200, q, 0),
                     lambda: _lib.rm_fp4_quantize_weight(p, 0, 2, 200, 30, w, 0),
                     lambda: _lib.rm_fp4_dequantize(q, 3, 200, p, 0, 200, 0),
                     lambda: _lib.rm_expert_sort(p, r, p, 1 << 20, 0),
                     lambda: _lib.rm_expert_gather(p, 0, r, p, 7, 8, 0),
                     lambda: _lib.rm_fp4_expert_gather(p, 0, r, q, 7, 200, 0),
                     lambda: _lib.rm_expert_combine(p, 0, r, None, p, 0, 7, 8, 0),
                     lambda: _lib.rm_expert_combine_backward(p, p, 0, r, p, p, p, 7, 8, 0)):
            try:
                call()
            except _lib.RankMixerError as e:
                assert e.status == _lib.RM_ERR_CUDA, e
            else:
                raise SystemExit("ran without a device")
    """, CUDA_VISIBLE_DEVICES="")
    assert got == ["rm:fp4_quantize", "rm:fp4_quantize_weight", "rm:fp4_dequantize", "rm:expert_sort", "rm:expert_gather",
                   "rm:fp4_expert_gather", "rm:expert_combine", "rm:expert_combine_backward"]


# ---- the tests' own restatements on values with known answers -------------------------------------

def test_the_reference_format():
    x = torch.zeros((7, 64))
    x[0, 3] = 6.0                                    # exactly the largest: scale 1
    x[1, 3], x[1, 40] = 6.0 * (1 + 2.0 ** -20), -24.0        # just above: scale 2; another block of its own
    x[2, 0], x[2, 33] = float("inf"), 1.0            # its block is NaN
    x[3, 0] = 2.0 ** -149                            # the smallest float: E = 1
    x[4, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.26])
    x[5, 0] = -0.0
    x[6, 0] = 3.0                                    # 3 is 6 with a scale of 1/2
    code, E = ref.quantise(x)
    assert E.tolist() == [[127, 127], [128, 129], [255, 125], [1, 127], [127, 127], [127, 127], [126, 127]]
    assert code[0, 0, 3] == 7 and code[1, 0, 3] == 5 and code[1, 1, 8] == 15 and code[2, 1, 1] == 6 and code[3, 0, 0] == 0
    assert code[4, 0, :16].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 8, 10, 10, 12, 12, 14, 14, 1]
    assert code[5, 0, 0] == 8 and code[6, 0, 0] == 7
    assert ref.packed(code)[4, :2].tolist() == [0x20, 0x42]


def test_the_reference_order_of_rows():
    G = torch.tensor([[[1.0, 0.0], [0.0, 2.0]], [[3.0, -1.0], [float("nan"), 0.5]], [[0.0, 4.0], [0.0, 0.0]]])   # [3, 2, 2]
    offsets, source, slot = ref.sorted_rows(G)
    assert offsets.tolist() == [0, 2, 3, 3, 5] and source.tolist() == [0, 2, 4, 1, 3]
    assert slot.tolist() == [[[0, -1], [-1, 3]], [[1, -1], [-1, 4]], [[-1, 2], [-1, -1]]]


def test_what_a_value_may_round_to():
    g = torch.tensor([[1.0, 2.5, 5.99, 0.26] + [0.0] * 28], dtype=torch.float64)
    q, lo, hi = ref.rounded_between(g, torch.full_like(g, 0.02))
    # the largest may be above 6, and the scale 2: 0.24 is then 0, and 5.97 and 6.01 are 6 by either scale
    assert q[0, :4].tolist() == [1.0, 2.0, 6.0, 0.5] and lo[0, :4].tolist() == [1.0, 2.0, 6.0, 0.0]
    assert hi[0, :4].tolist() == [1.0, 3.0, 6.0, 0.5]
