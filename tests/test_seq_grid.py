"""Launch limits of the sequence operators without a GPU: their grids
(tests/host/seq_grid_check.cpp) and the sizes that the entry points take."""
import ctypes
import os
import shutil
import subprocess

import pytest

from quantized_linear_recurrence_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_every_number_of_work_groups_has_a_grid(tmp_path):
    exe = tmp_path / "seq_grid_check"
    cmd = ["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           os.path.join(ROOT, "tests", "host", "seq_grid_check.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout[-3000:]


def test_sizes_at_the_limit(lores_lib):
    """The chunks' numbers, one grid row added, stay below 2^31."""
    n = ctypes.c_size_t(0)

    def status(T, B=65535, H=512):
        d = _lib.LoresScanDims(B, T, H, H, 32, 1, 0, 0)
        return lores_lib.lores_scan_workspace(ctypes.byref(d), 0, ctypes.byref(n))

    for B, H in ((65535, 512), (4096, 512), (65535, 1), (1, 512)):
        most = ((2 ** 31 - 2 ** 21 - 1) // H - 8) // B               # T / 32 + 8, rounded up
        T = 32 * (most - 8)
        if T > 2 ** 28:
            assert status(2 ** 28, B, H) == 0
            continue
        assert status(T, B, H) == 0
        assert status(T + 1, B, H) == _lib.LORES_EINVAL
        assert b"too large" in lores_lib.lores_last_error()
