"""The kernels that take more than 64 KB of LDS are allowed it on every device that
they are launched on, not only on the process's first: the built library, on a
stand-in for the HIP runtime that counts what each of two devices is told."""
import os
import subprocess
import sys

from bit_microscaled_quantized_amd import nvfp4 as nv

SHIM = r"""
#include <cstddef>
#include <cstdint>
extern "C" {
int device = 0, told[2] = {0, 0}, launched[2] = {0, 0}, fail = 0;
struct dim3_t { uint32_t x, y, z; };
int hipGetDevice(int *d) { *d = device; return 0; }
int hipFuncSetAttribute(const void *, int, int) { told[device]++; return fail; }
unsigned __hipPushCallConfiguration(dim3_t, dim3_t, size_t, void *) { return 0; }
int __hipPopCallConfiguration(dim3_t *, dim3_t *, size_t *, void *) { return 0; }
int hipLaunchKernel(const void *, dim3_t, dim3_t, void **, size_t, void *) { launched[device]++; return 0; }
int hipGetLastError() { return 0; }
}
"""

RUN = r"""
import ctypes, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # found before the runtime's own functions
from bit_microscaled_quantized_amd import nvfp4 as nv
device, fail = (ctypes.c_int.in_dll(shim, n) for n in ("device", "fail"))
told, launched = ((ctypes.c_int * 2).in_dll(shim, n) for n in ("told", "launched"))
A, BIG = 1 << 20, 1 << 34
calls = {
    "gemm": lambda: nv.nvfp4_gemm(64, 64, 64, A, A, A, A, A, 1, A, A, 64, 0.0, stream=0, raise_on_error=False),
    "gemm_bf16": lambda: nv.nvfp4_gemm_bf16(64, 64, 64, A, A, A, A, A, 1, A, A, 64, 0.0, stream=0,
                                            raise_on_error=False),
    "mxfp4": lambda: nv.mxfp4_gemm(128, 128, 128, A, A, A, A, A, 128, 0.0, stream=0, raise_on_error=False),
    "loss": lambda: nv.nvfp4_linear_cross_entropy(4, 100, 64, A, 64, A, 64, A, A, A, A, BIG, stream=0,
                                                  raise_on_error=False),
}
for name, call in calls.items():
    told[0] = told[1] = launched[0] = launched[1] = 0
    device.value, fail.value = 0, 1
    assert call() == nv.NVFP4_EHIP and launched[0] == 0, name
    fail.value = 0
    for d in (0, 1, 0, 1):
        device.value = d
        before = list(told)
        assert call() == nv.NVFP4_OK, (name, nv.NVFP4_OK)
        print(name, d, told[0] - before[0], told[1] - before[1], launched[0], launched[1], flush=True)
"""


def test_every_device_is_told(tmp_path):
    src, lib = tmp_path / "shim.cpp", tmp_path / "libshim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(nv.__file__)))
    r = subprocess.run([sys.executable, "-c", RUN, str(lib)], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    lines = [line.split() for line in r.stdout.splitlines()]
    assert len(lines) == 16, r.stdout
    for i, (name, d, told0, told1, launched0, launched1) in enumerate(lines):
        told = (int(told0), int(told1))
        if i % 4 == 0:  # device 0 again after its failure
            assert told[0] > 0 and told[1] == 0, lines[i]
        elif i % 4 == 1:  # the other device's first call
            assert told[1] > 0 and told[0] == 0, lines[i]
        else:
            assert told == (0, 0), lines[i]
        assert int(launched1 if d == "1" else launched0) > 0, lines[i]
