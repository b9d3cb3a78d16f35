"""What holds of the norm and rotation and of cross attention without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest

from precision_attention_fa4fp4_gb300 import api, build


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh"))))
def test_grids_that_start_early_load_plainly(name):
    """A kernel that starts while its predecessor runs reads what that writes: no load of it may need the memory
    unchanged from the kernel's start."""
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    if re.search(r"\b(wait_for_previous|grid_wait)\(", text) or name in ("cross.cuh", "cache_line.cuh"):
        assert not re.search(r"__ldg\b|__ldca|ld\.global\.nc|__restrict__", text)


TASKS = r"""
#include "rope.h"
#include <cstdio>
using namespace fa4;
// The tasks of the last warps of a grid of `ctas` CTAs with 8 warps, for `tokens` tokens in `parts` parts: each has to be
// in range, split into a part and a token as the kernel splits it, and the walks have to end at the count.
int main() {
  const long long cases[][3] = {{1 << 30, 2, 456}, {(1 << 30) - 1, 2, 456}, {(1 << 30) - 1000, 2, 456}, {1 << 30, 1, 304},
                                {1 << 29, 2, 456}, {2431, 4, 7}, {1, 2432, 304}};
  for (const auto& c : cases) {
    const Divisor by((int)c[0]);
    const unsigned long long all = (unsigned long long)c[0] * c[1];
    for (unsigned w = 0; w < c[2] * 8; w += 97) {
      unsigned long long want = w, seen = 0;
      for (Tasks t{w, (uint32_t)(c[2] * 8), (uint32_t)by.d * (int)c[1]}; t.more(); t.next(), want += c[2] * 8, ++seen) {
        const uint32_t n = t.now;
        const uint32_t q = (uint32_t)((((unsigned long long)n * by.m) >> 32) + n) >> by.s;
        if (t.now != want || want >= all || q != want / c[0] || (int)q >= c[1]) return printf("task %u of %llu\n", n, all), 1;
        if (seen > (1u << 21)) return printf("no end\n"), 1;
      }
      if (want < all) return printf("ends at %llu of %llu\n", want, all), 1;
    }
  }
  return 0;
}
"""


def test_tasks_of_the_largest_calls(tmp_path):
    """2^30 tokens with q and k are 2^31 tasks: all of them are gone through, and none behind them."""
    src = tmp_path / "tasks.cpp"
    src.write_text(TASKS)
    exe = str(tmp_path / "tasks")
    include = [os.path.join(build._cuda_home(), "include"), build.CSRC]
    subprocess.run(["g++", "-O1", "-std=c++17", *(x for i in include for x in ("-I", i)), str(src), "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    with open(os.path.join(build.CSRC, "rope.cu")) as f:
        assert f.read().count("Tasks task{") == 2          # both kernels count so


def test_no_query_heads_is_checked():
    """Without a query head dk and dv are still outputs: they are checked (here they are missing)."""
    build.build()
    lib = api.load_library()
    call = lambda Hkv, Nk: lib.fa4bf16_cross_bwd(  # noqa: E731
        None, None, None, None, None, None, None, 1, 0, Hkv, 4, Nk, 64, ctypes.c_float(0.0), None, None, None, None,
        ctypes.c_size_t(0), None)
    assert call(2, 8) == 1 and call(0, 8) == 0 and call(2, 0) == 0


def test_rows_are_counted_in_32_bits():
    """Sizes whose tasks would not be: refused before anything is looked at."""
    build.build()
    lib = api.load_library()
    for B, H, N, status in ((1 << 15, 64, 1 << 15, 2), (1 << 10, 1 << 20, 1 << 10, 2), (1 << 10, 1 << 19, 1 << 6, 1)):
        assert lib.fa4fp4_norm_rope(None, None, B, H, H, N, 64, None, None, None, None, None) == status
        assert lib.fa4fp4_norm_rope_bwd(None, None, 0, None, None, B, H, H, N, 64, None, None, None, None, None, None, None,
                                        ctypes.c_size_t(0), None) == status
