"""A workspace's size goes by the sizes of the call alone: queried with one GPU current and
used with another (fewer compute units, or none known) it is the one that the launch counts on.
The HIP runtime is a stand-in here; nothing is launched."""

import os
import shutil
import subprocess
import sys

import pytest

from int4_weight_only_amd import _lib

# a runtime whose device has as many compute units as the environment says
RUNTIME = r"""
#include <stdlib.h>
int hipGetDevice(int* device) { *device = 0; return 0; }
int hipDeviceGetAttribute(int* value, int attribute, int device) {
  *value = atoi(getenv("TEST_UNITS"));
  return *value > 0 ? 0 : 1;
}
"""

QUERY = """
import ctypes, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
i = ctypes.c_int64
for f in ("w4_bf16_moe_gemm_workspace", "w4_bf16_moe_wgrad_workspace", "w4_bf16_gemm_tn_workspace"):
    getattr(lib, f).restype = i
out = []
for M in (1, 2, 5, 70, 300, 1000, 2050, 8192):
    for N, K in ((64, 64), (64, 2048), (1024, 1024), (512, 8192), (4096, 4096), (2048, 80)):
        out.append(lib.w4_bf16_gemm_tn_workspace(i(M), i(N), i(K)))
        for k, E in ((1, 1), (4, 8)):
            out.append(lib.w4_bf16_moe_gemm_workspace(i(M), k, E, i(N), i(K), 64))
            out.append(lib.w4_bf16_moe_wgrad_workspace(i(M), k, E, i(N), i(K)))
print(*out)
"""


def test_sizes_do_not_go_by_the_current_device(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler for the stand-in of the runtime")
    source, shim = tmp_path / "runtime.c", tmp_path / "runtime.so"
    source.write_text(RUNTIME)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(shim), str(source)], check=True)

    def sizes(units):
        env = dict(os.environ, TEST_UNITS=str(units))
        r = subprocess.run([sys.executable, "-c", QUERY, str(shim), _lib.LIB_PATH], env=env, check=True,
                           capture_output=True, text=True)
        return r.stdout.split()
    many = sizes(256)
    assert any(int(n) > 0 for n in many) and any(int(n) == 0 for n in many)
    for units in (0, 32, 80, 304):
        assert sizes(units) == many, units
