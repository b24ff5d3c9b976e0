"""Where the cached attention's finishing kernel finds a row's sums
(row_pieces of hstu_cached.cuh), run on the host: for every way to cut a line
of work into parts the pieces that the cut leaves, and for records of any
content (what a workspace held before a call that gave up) nothing outside the
slots that exist."""
import os
import shutil
import subprocess

import pytest

from hstu_jagged_attention_02_gb300 import build as B

NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")

PROGRAM = r"""
#include <stdio.h>
#include <stdint.h>
#include <vector>
#include "hstu_cached.cuh"

using namespace hstu;

static uint32_t state = 12345u;
static uint32_t rnd() { state = state * 1664525u + 1013904223u; return state ^ (state >> 15); }

// Cuts the tiles of `cost` (far ones cost 2, near ones 6) of items in a line among CTAs of `quota`; a CTA takes the
// tiles that begin in its part.  Slot of a piece: item + CTA.
static int check_cut(const std::vector<std::vector<int>>& items, int H, int quota) {
  int64_t line = 0;
  int item = 0;
  for (const auto& tiles : items) {            // a block: H items of equal tiles
    int cost = 0;
    for (int c : tiles) cost += c;
    const int4 rec = make_int4((int)line, item, cost, 3 | (tiles.back() << 16));
    for (int h = 0; h < H; ++h) {
      int64_t at = line + (int64_t)h * cost, first = -1, lastc = -1, n = 0;
      for (int c : tiles) {
        const int64_t cta = at / quota;
        if (cta != lastc) { ++n; lastc = cta; if (first < 0) first = cta; }
        at += c;
      }
      const RowPieces r = row_pieces(rec, h, quota, 8, 1 << 30);
      if (r.n != n || r.slot != item + h + first) {
        printf("cut: item %d head %d: %lld pieces from %lld, not %lld from %lld\n", item, h, (long long)r.n,
               (long long)r.slot, (long long)n, (long long)(item + h + first));
        return 1;
      }
      // the last slot is the first that has to exist
      if (row_pieces(rec, h, quota, 8, r.slot + n).n != n || row_pieces(rec, h, quota, 8, r.slot + n - 1).n != 0) {
        printf("cut: the number of slots\n");
        return 1;
      }
    }
    line += (int64_t)H * cost;
    item += H;
  }
  return 0;
}

int main() {
  for (int round = 0; round < 3000; ++round) {
    const int H = 1 + rnd() % 5, near_cost = 5 + rnd() % 2, blocks = 1 + rnd() % 6;
    std::vector<std::vector<int>> items;
    for (int b = 0; b < blocks; ++b) {
      std::vector<int> t(rnd() % 9, 2);
      for (int k = rnd() % 5 + (t.empty() ? 1 : 0); k > 0; --k) t.push_back(near_cost);
      items.push_back(t);
    }
    if (check_cut(items, H, near_cost + rnd() % 40)) return 1;   // a CTA's part holds a tile's beginning
  }
  for (int round = 0; round < 20000000; ++round) {
    auto any = [&](int k) -> int { const int pick = rnd() % 6; const int v = (int)rnd();
      return pick == 0 ? v : pick == 1 ? (v & 0xffff) : pick == 2 ? (v & 0xff) : pick == 3 ? -(v & 0xfff) : pick == 4 ? 0x7fffffff - (v & k)
                                                                                                      : (int)0x80000000 + (v & k); };
    const int4 rec = make_int4(any(15), any(255), any(3), any(7));
    const int N = 8 << (rnd() % 5), quota = 1 + ((rnd() % 3) ? rnd() % 200 : rnd() % 2000000000u), h = rnd() % 32;
    const int64_t slots = 256 + rnd() % 100000;
    const RowPieces r = row_pieces(rec, h, quota, N, slots);
    if (r.n < 0 || (r.n > 0 && (r.slot < 0 || r.slot + r.n > slots || (rec.w & 0xffff) >= N))) {
      printf("record %d %d %d %d, quota %d: %lld pieces from %lld of %lld\n", rec.x, rec.y, rec.z, rec.w, quota,
             (long long)r.n, (long long)r.slot, (long long)slots);
      return 1;
    }
  }
  printf("ok\n");
  return 0;
}
"""


def test_a_rows_pieces(tmp_path):
    src, exe = tmp_path / "records.cu", tmp_path / "records"
    src.write_text(PROGRAM)
    r = subprocess.run([NVCC, *B.ARCH, *B.FLAGS, "-I", B.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
