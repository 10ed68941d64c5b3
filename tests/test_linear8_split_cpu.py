"""How the 8-bit linear layer shares its work out, without a GPU: the header's arithmetic, which the kernel for many tokens
runs too, compiled for the host."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_sparse_ffn_gb300", "csrc")

# Goes through what every cluster computes. Every step of every tile is done once; a tile that is done in parts is joined by
# exactly the clusters that have some of it, each of which left its part where the others look for it; no cluster has more
# than one part in a place; all tickets and places lie within the workspace.
WALK = r"""
#include <cstdio>
#include <vector>
#include "linear8_split.h"
using namespace sffn;

static long long bad(int tiles, int steps, int groups) {
  const L8Split w = l8_split(tiles, steps, groups);
  const int grid = w.whole ? w.groups : w.parted;
  if (grid < 1 || grid > groups || w.left < 0 || w.left >= groups || w.parted < w.left || w.parted > groups) return 1;
  std::vector<int> done(tiles), parts(tiles);
  for (int c = 0; c < grid; ++c) {
    L8Segments work(w, c);
    L8Segment s;
    int used[2] = {0, 0};
    while (work.next(w, s)) {
      if (s.tile < 0 || s.tile >= tiles || s.s0 < 0 || s.s1 <= s.s0 || s.s1 > steps) return 2;
      if (s.s0 > done[s.tile] ) return 3;   // clusters follow each other
      done[s.tile] += s.s1 - s.s0;
      if (s.part != (s.s1 - s.s0 < steps)) return 4;
      if (!s.part) continue;
      if (s.slot < 0 || s.slot > 1 || used[s.slot]++) return 5;
      const int left = s.tile - w.whole * w.groups;
      if (left < 0 || left >= w.left) return 6;
      const L8Sharers h = l8_sharers(w, left, c);
      if (h.from < 0 || h.to >= w.parted || h.from > c || h.to < c || h.from == h.to) return 7;
      ++parts[s.tile];
      for (int o = h.from; o <= h.to; ++o) {   // each of them has a part of the tile, where this one would look
        L8Segments other(w, o);
        L8Segment t;
        bool found = false;
        while (other.next(w, t)) found |= t.tile == s.tile && t.part && t.slot == l8_slot(w, left, o);
        if (!found) return 8;
      }
      if (c == h.to && parts[s.tile] != h.to - h.from + 1) return 9;   // arrivals that the last one has counted
    }
  }
  for (int t = 0; t < tiles; ++t)
    if (done[t] != steps) return 10;
  return 0;
}

int main() {
  long long wrong = 0;
  const int many[] = {74, 76, 80};
  for (int groups : many)
    for (int tiles = 1; tiles <= 2 * groups + 3; ++tiles)
      for (int steps = 1; steps <= 512; steps += steps < 128 ? 1 : 13) {
        const long long why = bad(tiles, steps, groups);
        if (why && ++wrong <= 5) printf("%d tiles of %d steps, %d clusters: %lld\n", tiles, steps, groups, why);
      }
  printf("%lld\n", wrong);
  return wrong != 0;
}
"""


def passes(program, tmp_path):
    src, exe = tmp_path / "program.cpp", tmp_path / "program"
    src.write_text(program)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_every_share_that_a_join_counts_has_steps(tmp_path):
    passes(WALK, tmp_path)


# Every number of outputs, inputs and tokens that a layer may have fits the blocks' shared memory.
FIT = r"""
#include <cstdio>
#include "linear8_split.h"
using namespace sffn;

int main() {
  long long wrong = 0;
  const int many[] = {148, 152, 160};
  for (int sms : many)
    for (int kp = 128; kp <= 65536; kp += 128)
      for (long long n = 1; n <= 1 << 20; n += n < 8192 ? 37 : n / 5) {
        const int most = l8_few_tokens((int)n, kp, sms);
        bool ok = most == 8 || most == 16 || most == 32;
        for (int tokens = 1; ok && tokens <= most; ++tokens) {
          const L8Few p = l8_few((int)n, kp, tokens, sms);
          const int rows = (int)((n + p.clusters - 1) / p.clusters), own = (kp / 64 + p.cs - 1) / p.cs * 64;
          ok = p.smem <= kL8FewSmem && p.clusters >= 1 && p.clusters <= n && rows <= kL8FewRows && 8 * p.nt >= tokens &&
               p.x_stride >= own && p.off_sum >= 8 * p.nt * own && p.off_sum % 16 == 0 &&
               p.smem >= p.off_sum + rows * 8 * p.nt * 4;
        }
        if (!ok && ++wrong <= 5) printf("%lld x %d, %d SMs, %d tokens a launch\n", n, kp, sms, most);
      }
  printf("%lld\n", wrong);
  return wrong != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_few_tokens_of_every_layer_fit(tmp_path):
    passes(FIT, tmp_path)


def test_warps_that_may_give_up_alone_do_not_wait_for_each_other_without_a_limit():
    """Between the kernel's first and last block barriers, which every thread meets, all waits are wait_for's."""
    with open(os.path.join(CSRC, "linear8_tc.cu")) as f:
        text = f.read()
    kernel = text[text.index("k_lin8_tc(const __grid_constant__"):text.index("__global__ void k_lin8_widen")]
    roles = kernel[kernel.index("fewer_registers<88>"):kernel.rindex("__syncwarp();")]
    assert roles.count("wait_for(") >= 8
    for name in ("__syncthreads", "cluster_sync_all", "_barrier(", "bar.sync", "mbar_try_wait", "while (true", "for (;;"):
        assert name not in roles, name
    assert "bar.sync" not in text
