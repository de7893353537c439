"""How the cross entropy's backward cuts its work up, checked on the CPU: the
host arithmetic of csrc/xent_plan.h, compiled alone.

Within a launch the MMA role hands over one accumulator per tile that has K
blocks, and the epilogue takes one per tile.  A tile without K blocks would
leave the epilogue waiting and every later tile one off."""
import random
import subprocess

import pytest

from _host_cxx import compile_host


# For each "T H V": the pieces, their slices, and commits and takes counted as
# the roles do; prints the plan, or what is wrong.
PLAN = r"""
#include <cstdio>
#include "xent_plan.h"
using namespace moe;
int main() {
  int T, H, V;
  while (std::scanf("%d %d %d", &T, &H, &V) == 3) {
    const XentBackwardPlan w = xent_backward_plan(T, H, V);
    const int tiles = xent_up(T, kXentTile) * xent_up(H, kXentTile);
    long long commits = 0, takes = 0, blocks = 0, want = 0;
    int pieces = 0, least = 1 << 30;
    const char* wrong = "";
    for (int v0 = 0; v0 < V; v0 += w.piece, ++pieces) {
      const int cols = V - v0 < w.piece ? V - v0 : w.piece;
      const int kblocks = xent_up(cols, kXentBK), ks = xent_piece_slices(w, cols);
      if (v0 == 0 && ks != w.slices) wrong = "the first piece does not write every slice";
      if (ks < 1 || ks > w.slices) wrong = "slices outside the workspace";
      for (int i = 0; i < ks; ++i) {
        const int k0 = xent_slice_start(kblocks, ks, i), k1 = xent_slice_start(kblocks, ks, i + 1);
        commits += (long long)tiles * (k1 > k0);
        takes += tiles;
        blocks += k1 - k0;
        if (k1 - k0 < least) least = k1 - k0;
      }
      want += kblocks;
      if (kblocks * kXentBK > xent_up(cols, kXentTile) * kXentTile) wrong = "K past the columns that dz holds";
    }
    if (blocks != want) wrong = "K blocks left out";
    std::printf("%d %d %lld %lld %d %s\n", pieces, w.slices, commits, takes, least, wrong);
  }
}
"""

# the last piece has fewer K blocks than the plan has slices
SHORT = [(4096, 1024, 32800), (4096, 256, 33000), (2048, 512, 65700), (8192, 1024, 16385), (4096, 2048, 32769),
         (4096, 2048, 32832), (2670, 768, 50257), (6144, 256, 65536), (1047, 1024, 128256), (7, 64, 2097152 + 100)]


def _plans(tmp_path, sizes):
    exe = compile_host(tmp_path, PLAN)
    text = "".join("%d %d %d\n" % s for s in sizes)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(sizes)
    for size, line in zip(sizes, out):
        pieces, slices, commits, takes, least, *wrong = line.split(maxsplit=5)
        yield size, int(pieces), int(slices), int(commits), int(takes), int(least), " ".join(wrong)


def test_every_tile_of_a_short_last_piece_has_its_accumulator(tmp_path):
    for size, pieces, slices, commits, takes, least, wrong in _plans(tmp_path, SHORT):
        assert pieces > 1 and slices > 1, size
        assert commits == takes and least >= 1 and not wrong, (size, wrong)


@pytest.mark.parametrize("seed", range(3))
def test_every_tile_has_its_accumulator(tmp_path, seed):
    rng = random.Random(seed)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())   # noqa: E731
    sizes = []
    for _ in range(4000):
        T, H = log(1, 1 << 17), 8 * log(1, 2048)
        piece = max(4096, (256 << 20) // (2 * max(T, 64)) // 256 * 256)
        V = rng.choice([log(1, 1 << 18), piece * rng.randint(1, 3) + rng.randint(0, 700)])
        sizes.append((T, H, V))
    several = 0
    for size, pieces, slices, commits, takes, least, wrong in _plans(tmp_path, sizes):
        several += pieces > 1 and slices > 1
        assert commits == takes and least >= 1 and not wrong, (size, wrong)
    assert several > 500
