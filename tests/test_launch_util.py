"""CPU test of the launch helpers (csrc/launch_util.cuh), as a host program on stand-ins for the device's
answers."""
import os
import shutil
import subprocess

import pytest

from structured_mask_linear_gb300 import _build

PROGRAM = r"""
#include <cuda_runtime.h>
#include <cstdio>
#include "launch_util.cuh"

#define HOLDS(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
  int asked = 0, n = -1;
  std::atomic<int> slot{0};
  auto fails = [&](int& v) { ++asked; v = 7; return cudaErrorMemoryAllocation; };
  auto answers = [&](int& v) { ++asked; v = 5; return cudaSuccess; };
  auto none = [&](int& v) { ++asked; v = 0; return cudaSuccess; };
  // an error is passed on and not kept
  HOLDS(ll::ask_once(&slot, n, fails) == cudaErrorMemoryAllocation && asked == 1);
  HOLDS(ll::ask_once(&slot, n, fails) == cudaErrorMemoryAllocation && asked == 2);
  // the next answer is, whatever would be answered later
  HOLDS(ll::ask_once(&slot, n, answers) == cudaSuccess && n == 5 && asked == 3);
  n = -1;
  HOLDS(ll::ask_once(&slot, n, fails) == cudaSuccess && n == 5 && asked == 3);
  // and one of 0 as well
  std::atomic<int> other{0};
  HOLDS(ll::ask_once(&other, n, none) == cudaSuccess && n == 0 && asked == 4);
  n = -1;
  HOLDS(ll::ask_once(&other, n, answers) == cudaSuccess && n == 0 && asked == 4);
  // without a place to keep it, it is asked every time
  HOLDS(ll::ask_once(nullptr, n, answers) == cudaSuccess && n == 5 && asked == 5);
  HOLDS(ll::ask_once(nullptr, n, none) == cudaSuccess && n == 0 && asked == 6);
  return 0;
}
"""


def test_only_answers_are_kept(tmp_path):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build._nvcc())))
    source, program = tmp_path / "ask.cpp", tmp_path / "ask"
    source.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", _build.CSRC, "-I", os.path.join(cuda, "include"), str(source), "-o", str(program)],
                   check=True)
    out = subprocess.run([str(program)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
