"""The look-up that every Linear's first call makes (csrc/tcgen05.cuh), made by several
threads at once: none may see it half done.  The driver's function is a stand-in that
takes its time, so the window is open on any machine; no GPU is used."""
import importlib.util
import os
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

static std::atomic<int> calls{0};
static cudaError_t slow_lookup(const char*, void** fn, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  std::this_thread::sleep_for(std::chrono::milliseconds(200));
  ++calls;
  *fn = reinterpret_cast<void*>(&slow_lookup);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define cudaGetDriverEntryPointByVersion slow_lookup
#include "tcgen05.cuh"

int main() {
  std::atomic<int> without{0}, ready{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&] {
      ++ready;
      while (ready < 8) std::this_thread::yield();
      if (!gbf::encode_fn()) ++without;
    });
  for (auto& t : threads) t.join();
  printf("%d %d\n", without.load(), calls.load());
}
"""


def test_every_thread_has_the_function(tmp_path):
    spec = importlib.util.spec_from_file_location("gbf_build", os.path.join(ROOT, "fusion_add_rmsnorm_gb300", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    try:
        cc = build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "first.cu", tmp_path / "first"
    src.write_text(PROGRAM)
    subprocess.run([cc, *build.ARCH, *build.FLAGS, "-I", build.CSRC, "-cudart", "static", str(src), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout
    assert out.split() == ["0", "1"], f"{out.split()[0]} of 8 threads without the function, {out.split()[1]} look-ups"
