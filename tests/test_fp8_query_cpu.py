"""What the FP8 launches ask the runtime once, as a host program of its own: a
failed query is not kept, and the register split is refused only where it does
not fit."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_quantized_rank_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "fp8_query.h"
using namespace cql;
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
  KeptAnswer kept;
  int asked = 0, n = -7;
  auto fails = [&](int& v) { ++asked; v = 0; return 3; };
  auto works = [&](int& v) { ++asked; v = 71; return 0; };
  CHECK(kept.get(n, fails) == 3 && asked == 1);
  CHECK(kept.get(n, fails) == 3 && asked == 2);           // asked again, not taken for the answer 0
  CHECK(kept.get(n, works) == 0 && n == 71 && asked == 3);
  n = 0;
  CHECK(kept.get(n, fails) == 0 && n == 71 && asked == 3);
  KeptAnswer zero;
  CHECK(zero.get(n, [&](int& v) { ++asked; v = 0; return 0; }) == 0 && n == 0 && asked == 4);
  CHECK(zero.get(n, works) == 0 && n == 0 && asked == 4); // 0 is an answer too
  // 512 threads that become 128 of 40, 128 of 104 and 256 of 176: 124 a thread
  const int sum = 128 * 40 + 128 * 104 + 256 * 176;
  for (int regs = 124; regs <= 128; ++regs) CHECK(register_split_fits(regs, 512, sum, 104));
  CHECK(!register_split_fits(123, 512, sum, 104) && !register_split_fits(96, 512, sum, 104));
  CHECK(!register_split_fits(96, 1024, sum, 104));        // a role cannot shrink to more than it has
  return 0;
}
"""


def test_queries(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "q.cpp", tmp_path / "q"
    src.write_text(PROGRAM)
    r = subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_pair_kernel_states_its_own_split():
    """The sum that is checked is the one that the kernel's roles ask for."""
    import re
    s = open(os.path.join(CSRC, "fp8_gemm.cu")).read()
    asked = [int(v) for v in re.findall(r"setmaxnreg\.\w+\.sync\.aligned\.u32 (\d+)", s)]
    assert asked == [40, 104, 176]                          # warps 0..3, 4..7, 8..15
    assert re.search(r"GM_REGS_SUM = 128 \* 40 \+ 128 \* 104 \+ 256 \* 176, GM_REGS_DEC = 104;", s)
    assert "GM_THREADS = 512" in s
