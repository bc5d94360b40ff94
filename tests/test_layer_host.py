"""The layer operators' host side without a GPU: csrc/lores_layer_api.cpp under
AddressSanitizer and UndefinedBehaviorSanitizer against stand-in launchers
(tests/host/layer_check.cpp), and the built library's refusals and workspaces."""
import ctypes
import os
import shutil
import subprocess

import pytest

from quantized_linear_recurrence_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_host_code_under_sanitizers(tmp_path):
    exe = tmp_path / "layer_check"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           os.path.join(ROOT, "quantized_linear_recurrence_amd", "csrc", "lores_layer_api.cpp"),
           os.path.join(ROOT, "tests", "host", "layer_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, (r.stdout[-3000:], r.stderr[-3000:])


def test_structures_have_the_header_s_layout():
    """Offsets as a C compiler lays out include/lores.h."""
    code = r'''
#include <stdio.h>
#include <stddef.h>
#include "lores.h"
#define P(s, f) printf("%zu ", offsetof(s, f));
int main(void) {
    P(lores_gated_dims, tokens) P(lores_gated_dims, heads) P(lores_gated_dims, per_head) P(lores_gated_dims, gate_first)
    P(lores_gated_dims, eps) P(lores_gated_dims, x_stride) P(lores_gated_dims, gate_stride)
    printf("%zu ", sizeof(lores_gated_dims));
    P(lores_block_dims, rows) P(lores_block_dims, act) P(lores_block_dims, scale) P(lores_block_dims, x_stride)
    P(lores_block_dims, gate_stride)
    printf("%zu %d %d %d %d\n", sizeof(lores_block_dims), LORES_MXFP4, LORES_ACT_NONE, LORES_ACT_SILU, LORES_ACT_SIGMOID);
    return 0;
}'''
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "t.c"), "w") as f:
            f.write(code)
        exe = os.path.join(d, "t")
        subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), f.name, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    g, b = _lib.LoresGatedDims, _lib.LoresBlockDims
    assert got == [g.tokens.offset, g.heads.offset, g.per_head.offset, g.gate_first.offset, g.eps.offset,
                   g.x_stride.offset, g.gate_stride.offset, ctypes.sizeof(g), b.rows.offset, b.act.offset,
                   b.scale.offset, b.x_stride.offset, b.gate_stride.offset, ctypes.sizeof(b), _lib.LORES_MXFP4,
                   _lib.LORES_ACT_NONE, _lib.LORES_ACT_SILU, _lib.LORES_ACT_SIGMOID]


def test_refusals_without_a_gpu(lores_lib):
    p, n = 0x100000, ctypes.c_size_t(0)
    d = _lib.LoresGatedDims(6, 4, 64, 0, 0, 0, 1, 0, 1e-6)
    d.x_stride[:] = d.gate_stride[:] = (256, 64)
    assert lores_lib.lores_gated_norm_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and 0 < n.value <= 24 * 64 * 4
    d.act = 9
    assert lores_lib.lores_gated_norm(ctypes.byref(d), p, p, p, 0, p, None, None) == _lib.LORES_EINVAL
    assert b"act must be" in lores_lib.lores_last_error()
    b = _lib.LoresBlockDims(6, 64, 0, 0, 0, 1e-6, 1.0, 64, 64, 64)
    assert lores_lib.lores_block_norm_workspace(ctypes.byref(b), ctypes.byref(n)) == 0 and 0 < n.value <= 12 * 64 * 4
    assert lores_lib.lores_block_norm(ctypes.byref(b), p, p, None, p, None, 0, p, None, p, None) == _lib.LORES_EINVAL
    assert lores_lib.lores_mx_quant(p, 48, 4, 48, 0, p, p, None) == _lib.LORES_EINVAL
    assert lores_lib.lores_mx_matmul(p, p, _lib.LORES_FP8, p, p, 4, 4, 64, _lib.LORES_FP32, p, None) == _lib.LORES_EINVAL
    assert b"LORES_BF16" in lores_lib.lores_last_error()
