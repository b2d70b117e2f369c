"""How paged attention shares its tiles out over CTAs, at the sizes the host accepts: the split's own
arithmetic, compiled for the host (no GPU, no launch)."""
from __future__ import annotations

import json
import os
import subprocess

import pytest

from fp8_quant_row_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "paged_attention_kernels.cuh"
using namespace fp8q;

// args: CTAs, tiles in all, whether a second round of CTAs has a tenth of them. Prints the CTAs whose first or last
// tile is found in another one.
template <int W>
void run(int grid, long long all, bool small) {
  AttnParams P{};
  P.grid = grid;
  AttnSplit s{kByTile, int((all + (long long)grid * W - 1) / ((long long)grid * W)), 0};
  if (small) s.rest = s.quota / 10, s.quota -= s.rest;
  int wrong = 0;
  for (int c = 0; c < (small ? 2 : 1) * grid; ++c) {
    const int64_t t0 = attn_begin<W>(P, s, c), t1 = attn_begin<W>(P, s, c + 1);
    if (t1 <= t0) { ++wrong; continue; }
    for (int64_t t : {t0, t0 + (t1 - t0) / 2, t1 - 1}) wrong += attn_cta<W>(P, s, t) != c;
  }
  std::printf("[%d, %d]", wrong, s.quota);
}
int main(int n, char** v) {
  const int grid = std::atoi(v[1]);
  const long long all = std::atoll(v[2]);
  if (std::atoi(v[4]) == 4) run<4>(grid, all, std::atoi(v[3])); else run<8>(grid, all, std::atoi(v[3]));
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "split.cu").write_text(PROGRAM)
    subprocess.run([_build.nvcc_path(), *_build.ARCH, "-std=c++17", "-cudart", "shared", f"-I{_build.INCLUDE}",
                    f"-I{_build.CSRC}", str(d / "split.cu"), "-o", str(d / "split"),
                    "-Xlinker", f"-rpath,{os.path.join(_build.CUDA_HOME, 'lib64')}"], check=True)

    def run(*args):
        out = subprocess.run([str(d / "split"), *map(str, args)], capture_output=True, text=True, timeout=60, check=True)
        return json.loads(out.stdout)

    return run


@pytest.mark.parametrize("grid,warps", [(152, 4), (152, 8), (304, 8), (456, 4)])
@pytest.mark.parametrize("tiles", [1 << 40, (1 << 40) - 12345, 1 << 38, 0xFFFFFFFF * 152, 10 ** 9, 77777])
@pytest.mark.parametrize("small", [0, 1])
def test_every_tile_is_found_in_its_cta(split, grid, warps, tiles, small):
    wrong, quota = split(grid, tiles, small, warps)
    assert wrong == 0, quota
    assert 0 < quota < 2 ** 31  # a warp's share, an int
