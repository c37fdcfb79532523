"""No exception passes the C boundary: with every allocation failing, the calls return their error (a C++
program whose operator new throws on demand, no GPU)."""
import os
import subprocess

import pytest

PROGRAM = r'''
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "moe.h"

static bool failing = false;
void* operator new(std::size_t n) {
  void* p = failing ? nullptr : std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void* operator new(std::size_t n, std::align_val_t a) {
  const std::size_t al = static_cast<std::size_t>(a);
  void* p = failing ? nullptr : std::aligned_alloc(al, (n + al - 1) / al * al);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p, std::align_val_t) noexcept { std::free(p); }
void operator delete(void* p, std::size_t, std::align_val_t) noexcept { std::free(p); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

int main() {
  moe_linear* l = moe_linear_create(300, 200);
  moe_plan* p = moe_plan_create(8, 2, 128, 128, 0, MOE_W_FP8);
  if (!l || !p) return 128;
  failing = true;
  int bad = 0;
  if (moe_linear_create(300, 200) || !strstr(moe_last_error(), "memory")) bad |= 1;
  if (moe_plan_create(8, 2, 128, 128, 0, MOE_W_FP8) || !strstr(moe_last_error(), "memory")) bad |= 2;
  if (moe_linear_create(0, 200) || !strlen(moe_last_error())) bad |= 4;
  if (moe_linear_set_weights(l, nullptr, nullptr) != MOE_ERR_INVALID_ARG || !strlen(moe_last_error())) bad |= 8;
  if (moe_linear_forward(l, l, MOE_BF16, 200, 4, l, MOE_BF16, 300, nullptr) != MOE_ERR_NOT_READY) bad |= 16;
  if (moe_route_logits(p, nullptr, 4, nullptr, nullptr, nullptr) != MOE_ERR_NOT_READY && !strlen(moe_last_error())) bad |= 16;
  if (moe_plan_create(8, 9, 128, 128, 0, MOE_W_FP8) || !strstr(moe_last_error(), "k=9")) bad |= 32;
  failing = false;
  moe_linear_destroy(l);
  moe_plan_destroy(p);
  l = moe_linear_create(300, 200);  // and the library still works
  if (!l || strlen(moe_last_error())) bad |= 64;
  moe_linear_destroy(l);
  return bad;
}
'''


def test_calls_return_when_memory_runs_out(tmp_path):
    from decode_batches_gb300 import LIB_PATH, build
    build.build()
    src = tmp_path / "alloc.cc"
    src.write_text(PROGRAM)
    libdir = os.path.dirname(LIB_PATH)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "lib64")
    exe = tmp_path / "alloc"
    r = subprocess.run(["g++", "-std=c++17", "-I", build.INCLUDE, str(src), "-o", str(exe), LIB_PATH, "-L", cuda, "-lcudart",
                        f"-Wl,-rpath,{libdir}:{cuda}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
