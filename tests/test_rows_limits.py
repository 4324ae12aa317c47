"""The many-row operators at the most rows a call takes, and what a call's first row
block must not reach (CPU: the packing of tiles; GPU: a projection of 2^24 rows)."""

import os
import subprocess

import pytest
import torch

from moe_decode_layer_gb300 import _lib, batch, build
from tests import rows_reference as ref

PACKING = r"""
#include <cstdio>
#include "rows_params.h"
using namespace moe::rows;
int main() {
  // a group may have all of a call's 2^24 rows, in tiles of 32 rows or more
  const long most = (1L << 24) / 32;
  const int groups[] = {0, 1, 511, kMaxGroups - 1}, rows[] = {1, 16, 255, kMaxN};
  const int firsts[] = {0, 1 << 24, (1 << 24) + 15 * kMaxAdapters};
  const long counts[] = {1, 32767, 32768, 32769, 65535, 65536, 131072, most};
  for (int g : groups) for (int n : rows) for (int p0 : firsts) for (long c : counts)
    for (long b : {0L, c / 2, c - 1}) {
      const int4 t = pack_tile(g, p0, n, (int)b, (int)c);
      if (tile_group(t) != g || tile_rows(t) != n || tile_first(t) != p0 || tile_block(t) != b || tile_blocks(t) != c) {
        std::printf("group %d rows %d first %d block %ld of %ld\n", g, n, p0, b, c);
        return 1;
      }
    }
  return 0;
}
"""


def test_tiles_of_the_largest_group(tmp_path):
    """What the plan writes for a tile is what the product reads, also for more than 32767 tiles of one group."""
    src, exe = tmp_path / "packing.cpp", tmp_path / "packing"
    src.write_text(PACKING)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, "-I", cuda, str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == ""


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [(1 << 22) + 129, 1 << 24])
def test_project_of_one_adapter_and_the_most_rows(rows):
    """More tiles of one adapter than 16 bits count; every row against the restatement."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, 8, generator=g, device="cuda").bfloat16()
    weight = torch.randn(8, 8, generator=g, device="cuda").bfloat16()
    ad = batch.Adapters(torch.randn(1, 8, 8, generator=g, device="cuda").bfloat16(),
                        torch.randn(1, 8, 8, generator=g, device="cuda").bfloat16())
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ids[5], ids[rows // 2] = -1, 1
    ws = torch.empty(batch.project_workspace(8, 8, rows, rank=8, num_adapters=1), dtype=torch.uint8, device="cuda")
    out = batch.project(x, weight, adapters=ad, adapter_ids=ids, workspace=ws)
    assert batch.status(ws) == _lib.MOE_OK
    for r in range(0, rows, 1 << 20):
        part = slice(r, r + (1 << 20))
        want, bound = ref.project(x[part], weight.double(), ad, ids[part])
        assert bool(((out[part].double() - want).abs() <= bound).all()), r
