"""The sequence operators' host side without a GPU: csrc/lores_seq_api.cpp under
AddressSanitizer and UndefinedBehaviorSanitizer against stand-in launchers
(tests/host/seq_check.cpp), and the built library's refusals and workspace."""
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
    exe = tmp_path / "seq_check"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           os.path.join(ROOT, "quantized_linear_recurrence_amd", "csrc", "lores_seq_api.cpp"),
           os.path.join(ROOT, "tests", "host", "seq_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, (r.stdout[-3000:], r.stderr[-3000:])


def _dims(**kw):
    d = _lib.LoresScanDims(2, 100, 4, 2, 64, 40, 1, 1)
    for n, v in kw.items():
        setattr(d, n, v)
    return d


def test_workspace_follows_the_shapes(lores_lib):
    """X and P as bf16 planes and six gates per token of a chunk; the backward
    pass adds the states and U, H in fp32, each piece rounded up to 256 bytes."""
    n = ctypes.c_size_t(0)

    def size(backward, **kw):
        assert lores_lib.lores_scan_workspace(ctypes.byref(_dims(**kw)), backward, ctypes.byref(n)) == 0
        return n.value

    units = 2 * 4 * 2                                # sequences, heads, chunks of 64
    tri = 3 * 32 * 32 * 2                            # three blocks of 32 x 32 on and below the diagonal
    assert size(0) == units * (3 * tri + 2 * tri + 6 * 64 * 4)
    assert size(0, delta=0) == units * (2 * tri + 6 * 64 * 4)
    assert size(1) == units * (6 * tri + 6 * 64 * 4 + 2 * 48 * (64 + 64) * 4)
    assert size(0, T=8) == 0 and size(1, T=8) > 0 and size(1, T=0) == 0
    assert size(0, in_bf16=0) == 2 * 4 * 4 * (6 * 32 * 32 * 2 + 6 * 32 * 4)   # chunks of 32


def test_refusals_without_a_gpu(lores_lib):
    p, n = 0x100000, ctypes.c_size_t(0)
    for kw in ({"B": 0}, {"T": -1}, {"H_k": 3}, {"d_k": 40}, {"d_v": 257}, {"delta": 2}):
        assert lores_lib.lores_scan_workspace(ctypes.byref(_dims(**kw)), 0, ctypes.byref(n)) == _lib.LORES_EINVAL
        assert lores_lib.lores_last_error()
    d = _dims()
    assert lores_lib.lores_scan(ctypes.byref(d), p, p, p, p, p, None, None, p, p, p, 16, None) == _lib.LORES_ESIZE
    assert lores_lib.lores_scan(ctypes.byref(d), None, p, p, p, p, None, None, p, p, p, 1 << 30, None) == _lib.LORES_EINVAL
    assert lores_lib.lores_rmsnorm(p, 8, None, 0, p, 0, 4, 0, 0, 1e-6, 0, p, None, None, None) == _lib.LORES_EINVAL
    assert b"n must be" in lores_lib.lores_last_error()
    assert lores_lib.lores_rmsnorm_workspace(4, 64, ctypes.byref(n)) == 0 and 0 < n.value <= 4 * 64 * 4
