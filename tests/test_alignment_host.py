"""Arrays of 32-bit values that are not aligned to them are refused on the host, before any launch (no GPU)."""
import os
import subprocess

import pytest

from test_rows_host import GOOD as ROWS, P
from test_verify_host import GOOD as VERIFY


@pytest.fixture(scope="module")
def lib():
    from decode_batches_gb300 import build, load_library
    build.build()
    return load_library()


@pytest.mark.parametrize("by", [1, 2, 3])
def test_row_moves_and_verification(lib, by):
    from decode_batches_gb300 import MOE_ERR_INVALID_ARG
    for name, good in ROWS.items():
        for key in ("inv", "w", "dw"):
            if key in good:
                assert getattr(lib, name)(*{**good, key: P + by}.values(), None) == MOE_ERR_INVALID_ARG, (name, key)
                assert b"aligned" in lib.moe_last_error()
    for key in ("drafts", "offsets", "u", "us", "tokens", "acc"):
        assert lib.moe_verify_drafts(*{**VERIFY, key: P + by}.values(), None) == MOE_ERR_INVALID_ARG, key
        assert b"aligned" in lib.moe_last_error()


PROGRAM = r'''
#include <cstdlib>
#include <cstring>
#include <cuda_runtime.h>

#include "moe.h"

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 4; return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n) { *p = std::calloc(n, 1); return cudaSuccess; }
cudaError_t cudaFree(void* p) { std::free(p); return cudaSuccess; }
cudaError_t cudaMemset(void* p, int v, size_t n) { std::memset(p, v, n); return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
}

int main() {
  moe_adapters* h = moe_adapters_create(4, 64, 96, 16, MOE_BF16);
  void* ws = std::aligned_alloc(256, 1 << 20);
  if (!h || moe_adapters_set_workspace(h, ws, 1 << 20, 1000) != MOE_OK) return 128;
  char* p = reinterpret_cast<char*>(4096);
  int bad = 0;
  for (int by = 1; by < 4; ++by) {
    const int32_t* ids = reinterpret_cast<const int32_t*>(p + by);
    if (moe_adapters_forward(h, p, 96, 4, ids, p, 64, p + 8192, MOE_FP32, 64, nullptr) != MOE_ERR_INVALID_ARG ||
        !strstr(moe_last_error(), "aligned"))
      bad |= 1 << by;
  }
  moe_adapters_destroy(h);
  return bad;
}
'''


def test_adapter_ids(tmp_path):
    """The handle needs memory before it takes a call: stand-ins for the CUDA runtime give it some."""
    from decode_batches_gb300 import LIB_PATH, build
    build.build()
    src, exe = tmp_path / "align.cc", tmp_path / "align"
    src.write_text(PROGRAM)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    lib64 = os.path.join(cuda, "lib64")
    r = subprocess.run(["g++", "-std=c++17", "-I", build.INCLUDE, "-I", os.path.join(cuda, "include"), str(src), "-o", str(exe),
                        LIB_PATH, "-L", lib64, "-lcudart", f"-Wl,-rpath,{os.path.dirname(LIB_PATH)}:{lib64}"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
