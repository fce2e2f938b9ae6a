"""RM_NVTX=1 puts every launch in a range: seen by an NVTX tool of a few lines, built here, that writes the names of the
ranges to a file."""
import os
import subprocess
import sys
import textwrap

import pytest

from rankmixer_feature_interaction_gb300 import build as rm_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOOL = r"""
#include <nvtx3/nvToolsExt.h>
#include <stdio.h>
#include <stdlib.h>
static int push(const char* name) {
    FILE* f = fopen(getenv("RANGES_LOG"), "a");
    if (f) fprintf(f, "%s\n", name), fclose(f);
    return 0;
}
int InitializeInjectionNvtx2(NvtxGetExportTableFunc_t get) {
    const NvtxExportTableCallbacks* c = (const NvtxExportTableCallbacks*)get(NVTX_ETID_CALLBACKS);
    NvtxFunctionTable table;
    unsigned int size;
    if (!c || !c->GetModuleFunctionTable(NVTX_CB_MODULE_CORE, &table, &size)) return 0;
    *table[NVTX_CBID_CORE_RangePushA] = (NvtxFunctionPointer)push;
    return 1;
}
"""


def ranges(tmp_path, body, **env):
    """The names of the ranges that `body` makes, in order."""
    (tmp_path / "tool.c").write_text(TOOL)
    include = os.path.join(os.path.dirname(os.path.dirname(rm_build.nvcc_path())), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-I", include, "-o", str(tmp_path / "tool.so"), str(tmp_path / "tool.c")],
                   check=True)
    log = tmp_path / "ranges"
    log.write_text("")
    env = {**os.environ, "PYTHONPATH": ROOT, "RM_NVTX": "1", "NVTX_INJECTION64_PATH": str(tmp_path / "tool.so"),
           "RANGES_LOG": str(log), **env}
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(body)], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return log.read_text().split()


def test_8bit_rows_and_weights_are_ranged(tmp_path):
    """Without a device: the launch fails, in its range."""
    got = ranges(tmp_path, """
        import ctypes
        from rankmixer_feature_interaction_gb300 import _lib
        buf = ctypes.create_string_buffer(1 << 16)
        p = (ctypes.addressof(buf) + 255) // 256 * 256
        q = _lib.rm_fp8_tensor(p, p + 4096, 208, 4, _lib.RM_E4M3)
        for call in (lambda: _lib.rm_fp8_quantize(p, 0, 3, 200, 200, q, 0),
                     lambda: _lib.rm_fp8_quantize_weight(p, 0, 2, 3, 200, q, 0),
                     lambda: _lib.rm_fp8_dequantize(q, 3, 200, p, 0, 200, 0)):
            try:
                call()
            except _lib.RankMixerError as e:
                assert e.status == _lib.RM_ERR_CUDA, e
            else:
                raise SystemExit("ran without a device")
    """, CUDA_VISIBLE_DEVICES="")
    assert got == ["rm:fp8_quantize", "rm:fp8_quantize_weight", "rm:fp8_dequantize"]


@pytest.mark.gpu
def test_8bit_ffn_is_ranged(tmp_path):
    got = ranges(tmp_path, """
        import torch
        from rankmixer_feature_interaction_gb300 import api
        W1, W2 = torch.ones((2, 32, 64), device="cuda"), torch.ones((2, 64, 32), device="cuda")
        m = api.Fp8PFFN(W1, torch.zeros((2, 64), device="cuda"), W2, torch.zeros((2, 32), device="cuda"))
        X = torch.ones((5, 2, 32), device="cuda")
        m.forward(X)
        V, kept = m.forward_train(X)
        m.backward(X, kept)
        api.fp8_wgrad(kept["x"], X.to(torch.bfloat16))
        api.fp8_matmul(kept["x"], m.W1)
    """)
    forward = ["rm:fp8_quantize", "rm:fp8_product", "rm:fp8_product"]
    assert got == ["rm:fp8_quantize_weight"] * 2 + forward * 3 + ["rm:fp8_wgrad"] * 3 + ["rm:fp8_product"]
