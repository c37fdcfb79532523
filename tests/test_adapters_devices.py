"""A handle of adapters and two devices: a C++ program whose own CUDA runtime calls stand in for the library's (no GPU).  The
handle's calls are for the device that holds its memory; with another one current they are refused before they touch it."""
import os
import subprocess

PROGRAM = r'''
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <cuda_runtime.h>

#include "moe.h"

static int current = 0, synced[2] = {0, 0}, copies = 0;
static const int sms[2] = {4, 200};
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = current; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) { *v = sms[d]; return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n) { *p = std::calloc(n, 1); return cudaSuccess; }
cudaError_t cudaFree(void* p) { std::free(p); return cudaSuccess; }
cudaError_t cudaMemset(void* p, int v, size_t n) { std::memset(p, v, n); return cudaSuccess; }
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) { ++copies; std::memcpy(d, s, n); return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { ++synced[current]; return cudaSuccess; }
}

int main() {
  int bad = 0;
  uint32_t code = 7;
  moe_adapters* h = moe_adapters_create(4, 64, 96, 16, MOE_BF16);   // the first device is current
  if (!h) return 128;
  if (moe_adapters_get_device_error(h, &code) != MOE_OK || code) bad |= 1;   // no memory yet: any device will do
  const size_t small = moe_adapters_workspace_bytes(h, 1000);
  static char* ws = static_cast<char*>(std::aligned_alloc(256, 1 << 20));
  current = 1;
  // the memory goes to the second device, whose SMs count: the first one's workspace may be too small
  if (moe_adapters_set_workspace(h, ws, small, 1000) != MOE_ERR_WORKSPACE) bad |= 2;
  const size_t large = moe_adapters_workspace_bytes(h, 1000);
  if (large <= small || large > (1 << 20)) bad |= 4;
  if (moe_adapters_set_workspace(h, ws, large, 1000) != MOE_OK) bad |= 8;
  current = 0;
  const int before = synced[0] + copies;
  code = 7;
  if (moe_adapters_get_device_error(h, &code) != MOE_ERR_INVALID_ARG || !strstr(moe_last_error(), "device")) bad |= 16;
  if (synced[0] + copies != before) bad |= 32;
  if (moe_adapters_set_workspace(h, ws, large, 1000) != MOE_ERR_INVALID_ARG) bad |= 64;
  current = 1;
  if (moe_adapters_get_device_error(h, &code) != MOE_OK || code) bad |= 16;
  moe_adapters_destroy(h);
  return bad;
}
'''


def test_calls_with_another_device_current(tmp_path):
    from decode_batches_gb300 import LIB_PATH, build
    build.build()
    src = tmp_path / "devices.cc"
    src.write_text(PROGRAM)
    libdir = os.path.dirname(LIB_PATH)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    lib64, exe = os.path.join(cuda, "lib64"), tmp_path / "devices"
    r = subprocess.run(["g++", "-std=c++17", "-I", build.INCLUDE, "-I", os.path.join(cuda, "include"), str(src), "-o", str(exe),
                        LIB_PATH, "-L", lib64, "-lcudart", f"-Wl,-rpath,{libdir}:{lib64}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)


def test_a_workspace_on_another_device_is_refused(monkeypatch):
    import pytest
    import torch

    import decode_batches_gb300 as p

    class Elsewhere:                       # a buffer as a second device would have it
        device, is_cuda, dtype = "cuda:1", True, torch.uint8
        get_device = staticmethod(lambda: 1)
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: 1 << 20)
        numel = staticmethod(lambda: 1 << 20)
        element_size = staticmethod(lambda: 1)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    ad = p.LowRankAdapters(4, 64, 96, 16)
    with pytest.raises(ValueError, match="current CUDA device"):
        ad.set_workspace(Elsewhere(), 100)
    assert ad.T_max == 0
