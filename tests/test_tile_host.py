"""Host-side arithmetic of the dense products' tile (csrc/linear_tile.h), as constant expressions: an undefined
operation in one is a compile error.  Nothing runs on a GPU."""
import os
import subprocess

import pytest

from grouped_gemm_top_amd import build as B

CODE = r"""
#include "linear_tile.h"
using moe::ln::k_slice;
using moe::ln::KSlice;

// the slices follow each other from 0 to the end, and each knows its term and its step within it
constexpr bool covers(int terms, int steps, int S) {
  int at = 0;
  for (int s = 0; s < S; ++s) {
    const KSlice q = k_slice(terms, steps, s, S);
    if (q.n < 0) return false;
    if (q.n > 0 && (q.term < 0 || q.term >= terms || q.step < 0 || q.step >= steps || q.term * steps + q.step != at))
      return false;
    at += q.n;
  }
  return at == terms * steps;
}
constexpr bool all() {
  for (int terms = 1; terms <= 6; terms += 5)
    for (int steps = 0; steps <= 9; ++steps)
      for (int S = 1; S <= 64; S *= 2)
        if (!covers(terms, steps, S)) return false;
  return true;
}
static_assert(all(), "");
static_assert(k_slice(6, 0, 3, 4).n == 0, "no step where nothing is summed over");
static_assert(covers(6, (1 << 22) + 1, 64), "");
"""


def test_slices_of_a_contraction(tmp_path):
    """Among them those of a sum over no token at all, which a device-side count can give."""
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not found")
    src = tmp_path / "slices.hip"
    src.write_text(CODE)
    r = subprocess.run([B.HIPCC, *B.FLAGS, "--offload-host-only", "-fsyntax-only", str(src)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
