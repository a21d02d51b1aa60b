"""Kernels whose LDS grows with a row's width are allowed their most once on every device, and
that never changes: calls of other widths, on other host threads among them, cannot take it
away between the setting and the launch.  The built library, on a stand-in for the HIP runtime
that keeps each kernel's limit and checks every launch against it."""
import os
import subprocess
import sys

import pytest

from bit_microscaled_quantized_amd import nvfp4 as nv

SHIM = r"""
#include <cstddef>
#include <cstdint>
#include <map>
#include <utility>
extern "C" {
int device = 0, told = 0, changed = 0, above = 0, large = 0, launched = 0, fail = 0;
struct dim3_t { uint32_t x, y, z; };
static std::map<std::pair<int, const void *>, int> limit;
static struct { dim3_t grid, block; size_t shmem; void *stream; } config;
int hipGetDevice(int *d) { *d = device; return 0; }
int hipFuncSetAttribute(const void *f, int, int value) {
  if (fail) return fail;
  told++;
  auto it = limit.find({device, f});
  changed += it != limit.end() && it->second != value;
  limit[{device, f}] = value;
  return 0;
}
unsigned __hipPushCallConfiguration(dim3_t grid, dim3_t block, size_t shmem, void *stream) {
  config = {grid, block, shmem, stream};
  return 0;
}
int __hipPopCallConfiguration(dim3_t *grid, dim3_t *block, size_t *shmem, void **stream) {
  *grid = config.grid, *block = config.block, *shmem = config.shmem, *stream = config.stream;
  return 0;
}
int hipLaunchKernel(const void *f, dim3_t, dim3_t, void **, size_t shmem, void *) {
  launched++;
  if (shmem <= 64 * 1024) return 0;
  large++;
  auto it = limit.find({device, f});
  above += it == limit.end() || shmem > (size_t)it->second;
  return 0;
}
int hipGetLastError() { return 0; }
}
"""

RUN = r"""
import ctypes, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # found before the runtime's own functions
from bit_microscaled_quantized_amd import nvfp4 as nv
device, told, changed, above, large, launched, fail = (
    ctypes.c_int.in_dll(shim, n) for n in ("device", "told", "changed", "above", "large", "launched", "fail"))
A, BIG = 1 << 20, 1 << 34


def block_norms(dt, gate, rows, cols):
    return nv.nvfp4_block_norms_backward(
        A, A, A, A, None if gate is None else A, dt, rows, cols, cols, cols, cols, cols, cols if gate == "token" else 0, 0,
        A, A, 0, A, A, 1.0, A, cols, A, cols, None, cols, A, A, A, BIG, stream=0, raise_on_error=False)


def rms_norm(dt, gate, rows, cols):
    return nv.nvfp4_rms_norm_backward(A, A, A, dt, rows, cols, cols, cols, cols, A, dt, A, 0.0, 0, A, cols, A, cols, A, A,
                                      BIG, stream=0, raise_on_error=False)


call = dict(block_norms=block_norms, rms_norm=rms_norm)[sys.argv[2]]
kinds = [(dt, gate) for dt in (0, 1) for gate in ((None, "channel", "token") if call is block_norms else (None,))]
# every eighth part of the widths that a workgroup's registers hold, up and down; few rows, and so many that they stream
widths = list(range(1024, 32769, 1024))
sizes = [(rows, cols) for cols in widths + widths[::-1] for rows in (3, 700, 40000)]
fail.value = 1  # a kernel that could not be allowed its LDS is not launched, and is told again
failed = [(dt, gate, rows, cols) for dt, gate in kinds for rows, cols in sizes if call(dt, gate, rows, cols) != nv.NVFP4_OK]
assert failed and above.value == 0 and large.value == 0
fail.value = 0
for d in (0, 1, 0):
    device.value = d
    before = told.value
    for dt, gate in kinds:
        for rows, cols in sizes:
            assert call(dt, gate, rows, cols) == nv.NVFP4_OK, (dt, gate, rows, cols)
    print(d, told.value - before, changed.value, above.value, large.value, launched.value, flush=True)
"""


@pytest.mark.parametrize("name", ["block_norms", "rms_norm"])
def test_limits_are_set_once(tmp_path, name):
    src, lib = tmp_path / "shim.cpp", tmp_path / "libshim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(nv.__file__)))
    r = subprocess.run([sys.executable, "-c", RUN, str(lib), name], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    lines = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
    assert [line[0] for line in lines] == [0, 1, 0]
    for d, told, changed, above, large, launched in lines:
        assert changed == 0, "a kernel's limit was set to another value"
        assert above == 0, "a launch beyond the kernel's limit"
        assert large > 0 and launched > large
    assert lines[0][1] > 0 and lines[1][1] == lines[0][1], "a device was told less than the other"
    assert lines[2][1] == 0, "a device was told again"
