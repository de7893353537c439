// xent_plan.h - how the cross entropy's backward cuts its work up (xent.cu).
// Host arithmetic, and the one division that host and kernels share; no CUDA
// header, so that it can be checked without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define XENT_HD __host__ __device__ __forceinline__
#else
#define XENT_HD inline
#endif

namespace moe {

constexpr int kXentTile = 256;                  // rows and columns of an output tile
constexpr int kXentBK = 64;                     // K elements per stage
constexpr int kXentSplitRows = 32;              // most tokens whose dz is kept as two bf16 numbers

inline int xent_up(int64_t a, int b) { return (int)((a + b - 1) / b); }
inline size_t xent_align(size_t x) { return (x + 255) & ~(size_t)255; }

// The backward's pieces of the vocabulary: [T, piece] of dz in bf16 is held
// to about 256 MB, and a piece to whole tiles.  Up to 32 tokens (whose 64 rows
// fill one K block and a part of one row tile all the same) it is kept as a sum
// of two bf16 numbers: where one target's rounding is most of an output's error,
// it could be twice that of the output's own rounding (one token, V = 1000:
// 0.0030 against 0.0019 relative).  Over all rows of 64 tokens and more that
// comes to 0.0020; a row of dX alone is as far off as before, and so are both
// outputs of a long batch in which only a few rows count, since the number of
// those is not known here.  The second half costs 3 us of 18 at 7 x 512,
// V = 5000, and 18 of 129 at 32 x 2048, V = 32000; among many tokens it would
// double the products of dX and dW.
struct XentBackwardPlan {
  size_t dz, acc, total;   // workspace: dz [rows][piece] bf16, dX's sums [slices][rows][Hp] fp32
  int piece, slices, Hp, rows;
};
inline XentBackwardPlan xent_backward_plan(int T, int H, int V) {
  XentBackwardPlan w;
  const int vp = xent_up(V, kXentTile) * kXentTile;
  w.rows = T <= kXentSplitRows ? 2 * kXentSplitRows : T;
  int64_t piece = (256LL << 20) / (2 * (int64_t)w.rows) / kXentTile * kXentTile;
  if (piece < 4096) piece = 4096;
  w.piece = piece < vp ? (int)piece : vp;
  w.Hp = xent_up(H, kXentTile) * kXentTile;
  // few dX tiles: their K (the piece) is cut into slices until every SM pair
  // has two tiles; a slice keeps at least 512 columns
  const int tiles = xent_up(T < 1 ? 1 : T, kXentTile) * xent_up(H, kXentTile);
  int ks = xent_up(152, tiles);
  if (ks > w.piece / 512) ks = w.piece / 512;
  w.slices = ks < 1 ? 1 : ks;
  size_t o = 0;
  w.dz = o; o += xent_align((size_t)w.rows * w.piece * 2);
  w.acc = o; o += xent_align((size_t)w.slices * w.rows * w.Hp * sizeof(float));
  w.total = o ? o : 256;
  return w;
}

// Slices of dX's K in a piece of `cols` columns: every one has at least one K
// block, because a tile without K would have no accumulator to hand over.  A
// short last piece takes fewer than the plan's: it only adds to the sums that
// the first piece, which always has them all, has written.
inline int xent_piece_slices(const XentBackwardPlan& w, int cols) {
  const int kblocks = xent_up(cols, kXentBK);
  return w.slices < kblocks ? w.slices : kblocks;
}

// K blocks [result, that of i + 1) of slice i of ks.
XENT_HD int xent_slice_start(int kblocks, int ks, int i) { return (int)((int64_t)kblocks * i / ks); }

}  // namespace moe
