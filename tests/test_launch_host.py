"""CPU checks of the launches' host side: a program of the header's functions with stand-ins for
CUDA's."""
import os
import subprocess

from tiled_top_sparse_gb300 import _build

PROGRAM = r"""
#include "launch.cuh"
int main() {
  std::atomic<int> known{0};
  int asked = 0, value = -1;
  auto fails = [&](int*) { ++asked; return cudaErrorMemoryAllocation; };
  auto works = [&](int* n) { ++asked; *n = 168; return cudaSuccess; };
  if (tts::ask_once(known, &value, fails) != cudaErrorMemoryAllocation) return 1;
  if (tts::ask_once(known, &value, fails) != cudaErrorMemoryAllocation || asked != 2) return 2;
  if (tts::ask_once(known, &value, works) != cudaSuccess || value != 168 || asked != 3) return 3;
  value = -1;
  if (tts::ask_once(known, &value, fails) != cudaSuccess || value != 168 || asked != 3) return 4;
  return 0;
}
"""


def test_a_failed_query_is_asked_again(tmp_path):
    """A kernel's registers are asked for once; a query that fails for a passing reason returns its
    error and does not stay."""
    src, exe = tmp_path / "ask.cu", tmp_path / "ask"
    src.write_text(PROGRAM)
    r = subprocess.run([_build._nvcc(), *_build.ARCH, "-std=c++17", "-I", _build.CSRC, str(src), "-o",
                        str(exe)], capture_output=True, text=True, env=dict(os.environ))
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)]).returncode == 0
