// xent.cu - softmax cross entropy over a large vocabulary, straight from the
// hidden states, forward and backward.
//
//   z = X W^T                          X [T, H], W [V, H], z never stored
//   lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target
//   dz = exp(z - lse_t) - onehot(target),  dX = s dz W,  dW = s dz^T X
//
// The forward is one GEMM whose epilogue reduces each 256 x 256 logit tile to
// a maximum and a sum per row (an online softmax, 8 bytes per row and 128
// columns instead of 512 bytes of logits); a second kernel joins the pieces.
// The backward goes through the vocabulary in pieces: it forms the piece's
// logits again, turns them into dz in the epilogue (bf16, [T, piece]) and
// multiplies that by the piece's weights (added to dX's fp32 sums) and by X
// (the piece's rows of dW).  Products: 2 T V H flops forward, 6 T V H
// backward, which is what bounds it for T in the hundreds and more; for a few
// tokens the bound is reading W.
//
// GEMM structure (as the expert engine in gemm.cu): persistent SM pairs
// (clusters of two CTAs, cta_group::2 tcgen05 MMAs of 256 x 256 x 16), TMA
// loads into a ring of 64-element K stages, two TMEM accumulators so that one
// tile's epilogue runs under the next tile's MMAs.  An accumulator truncates
// what it adds, towards 0: over 4096 columns of K the log sum came out 2e-5 too
// small on average, over 512 2.4e-6, which is what rounded fp32 sums lose.  The
// forward therefore adds its logits up in fp32 registers from segments of up to
// 512 columns, one accumulator each.  (T = 2000, H = 4096, V = 32768: the losses
// are 2e-7 off their 64-bit values, 4e-7 with segments of 1024 columns, 2e-6 with
// whole tiles.  It costs 6% of the forward at T = 16384, H = 2048, V = 65536 and
// 1% of a training step; segments of 1024 half that; of 256 20%, since an
// epilogue then takes longer than a segment.)  The backward's exponentials are
// rounded to bf16 and keep whole tiles.
//
// Warp 0 loads A, warp 1 issues the MMAs, warps 2..9 are the epilogue (two per
// TMEM lane quarter, 128 columns each: an exponential per logit is too much for
// four warps), warp 10 loads B.  Every wait is bounded, as there.
//
// Measured (GB300): forward at T = 16384, H = 2048, V = 65536 2.8 ms (1.57
// PFLOP/s); forward and backward at T = 8192, H = 4096, V = 131072 21.8 ms (1.61
// PFLOP/s of the 8 T V H products; a library's plain bf16 products sustain 1.70
// under the power cap); tensor pipe 86 - 90% busy in the backward.  H = 2048, V =
// 32000, where reading W takes 19 us and writing dW as long again: forward of 17
// to 256 tokens 38 - 43 us (nearly empty tiles, two rounds over the SM pairs),
// backward of 1 to 32 tokens 118 - 132, of 33 to 256 111 - 127 (W is read for the
// logits and again for dX, in launches of their own).  Pieces of
// 256 MB of dz: 64 MB are 8% slower (more adds to dX), 512 MB 1% faster.
// Sweeps of 8 m-tiles over n: 4, 16 and 32 are 1 - 2% slower.
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "staging.h"
#include "xent_plan.h"

namespace moe {

namespace {

constexpr int kStages = 6;
constexpr int kBK = kXentBK;                    // K elements per stage
constexpr int kABytes = 128 * 128;              // 128 rows x 64 bf16
constexpr int kStageBytes = 2 * kABytes;        // a CTA's A rows and its half of B
constexpr int kAtomBytes = kBK * 128;           // 64 K rows x 64 MN elements (MN-major box)
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps + 32;
constexpr int kStgBytes = kEpiWarps * 4096;     // two 32 x 32 bf16 boxes per epilogue warp
constexpr int kSmemBytes = kStages * kStageBytes + kStgBytes + 1024 + 256;
constexpr int kTile = kXentTile;
constexpr int kSegment = 8;                     // most K blocks that the forward adds up in one accumulator
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFewTokens = 16;                  // most tokens of the kernel for few tokens
constexpr int kFewMaxBlocks = 512;
constexpr int kSplitRows = kXentSplitRows;
static_assert(2 * kSplitRows == kBK, "both parts are one K block of dW");
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

enum : int { XK_STATS = 0, XK_DZ = 1, XK_DX = 2, XK_DW = 3 };

// One GEMM of a launch.  Operand coordinates are the tile's plus an origin.
struct XJob {
  CUtensorMap tmA, tmB, tmO;
  int kind;
  int a_mn, b_mn;        // operand stored M-/N-major (1) or K-major (0)
  int tn;                // tile width (MMA N): 256, or 192 (K-major B)
  int mt, nt, ks;        // 256-row tiles, tn-column tiles, slices of K
  int kblocks;           // 64-element K blocks of the whole K
  int group;             // m-tiles that share one sweep over the n-tiles
  int b_n0, b_k0;        // origins of B (a piece of the vocabulary)
  int out_m0;            // first output row (DW)
};

struct XParams {
  XJob job[2];
  int njob;
  int catch_up;          // tiles of job 1 that weigh as much as one of job 0
  int T, H, V;
  // targets and statistics
  const void* targets;
  int index64, ignore_index;
  const float* lse;
  const float* dloss;
  const float* total;    // {sum, mean, count}
  int reduction;
  int segment;           // STATS: K blocks per accumulator
  // outputs
  float2* part;          // STATS: [2 nt][T] {max, sum} in the log2 domain
  float* zt;             // STATS: [T] target logits times log2(e)
  unsigned* ticket;      // STATS: zeroed for the join kernel
  float* acc;            // DX: fp32 sums [ks][T][Hp]
  int zcols;             // DZ: columns of the dz buffer
  int split;             // dz as a sum of two bf16 numbers: rows 0..31 and 32..63
  int rows;              // rows of dz and of dX's sums: T, or 64 if split
  int Hp;
  int add, last;         // DX: add to acc; write bf16 results
  int32_t* status;
  unsigned long long wait_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Target of a row: its column, -1 if the row is ignored, -2 if it is outside
// [0, V) (the caller reports it and treats the row as ignored).
__device__ __forceinline__ int target_of(const void* targets, int index64, int ignore, int V, int row) {
  const long long t = index64 ? static_cast<const long long*>(targets)[row]
                              : (long long)static_cast<const int32_t*>(targets)[row];
  if (t == ignore) return -1;
  return t >= 0 && t < V ? (int)t : -2;
}

// The tiles of one SM pair, in the order that all of its roles follow.  The
// first job's tiles go round the pairs; where its last round leaves some pairs
// without a tile, those first take as many of the second job's tiles as weigh
// as much (`catch_up`), and the rest goes round all pairs, theirs first.
// (Against going round regardless: 1% of the whole step at T = 8192, H = 4096,
// V = 131072, 2% at T = 4096, H = 2048, V = 50001.)
struct Schedule {
  int pair, pairs, n0, n1, own0, short_from, shared, catch_up;
  __device__ __forceinline__ Schedule(const XParams& P) {
    pair = blockIdx.x / 2;
    pairs = gridDim.x / 2;
    n0 = P.job[0].mt * P.job[0].nt * P.job[0].ks;
    n1 = P.njob > 1 ? P.job[1].mt * P.job[1].nt * P.job[1].ks : 0;
    own0 = pair < n0 ? (n0 - 1 - pair) / pairs + 1 : 0;
    short_from = n0 % pairs;               // pairs from here on have a tile less (0: none has)
    shared = short_from ? P.catch_up * (pairs - short_from) : 0;
    catch_up = pair >= short_from && short_from ? P.catch_up : 0;
  }
  // The k-th tile: its number over both jobs, or -1 past the last.
  __device__ __forceinline__ int tile(int k) const {
    if (k < own0) return pair + k * pairs;
    k -= own0;
    int i;
    if (k < catch_up) {
      i = k * (pairs - short_from) + pair - short_from;
    } else {
      i = pair - short_from;
      i = shared + (i < 0 ? i + pairs : i) + (k - catch_up) * pairs;
    }
    return i < n1 ? n0 + i : -1;
  }
};

struct XTile {
  int p, kind, m0, n0, ntile, slice, kb0, kb1;
};

__device__ __forceinline__ XTile decode(const XParams& P, const Schedule& sc, int t, int rank) {
  const int p = t >= sc.n0;
  const XJob& g = P.job[p];
  int lt = t - (p ? sc.n0 : 0);
  XTile ti;
  ti.p = p;
  ti.kind = g.kind;
  ti.slice = lt / (g.mt * g.nt);
  lt -= ti.slice * g.mt * g.nt;
  const int gi = lt / (g.group * g.nt);
  const int r = lt - gi * g.group * g.nt;
  const int gm = min(g.group, g.mt - gi * g.group);
  ti.ntile = r / gm;
  ti.m0 = (gi * g.group + (r - ti.ntile * gm)) * kTile + rank * 128;
  ti.n0 = ti.ntile * g.tn;
  ti.kb0 = xent_slice_start(g.kblocks, g.ks, ti.slice);
  ti.kb1 = xent_slice_start(g.kblocks, g.ks, ti.slice + 1);
  return ti;
}

// Loads A (part 0, which also arms the leader's full barrier) or B (part 1)
// of every stage: this CTA's 128 rows of A and its half of the tile's B columns.
__device__ void load_role(const XParams& P, const Schedule& sc, int rank, uint8_t* stages,
                          uint64_t* full, uint64_t* empty, const WaitCtl& wc, int part) {
  int it = 0;
  bool ok = true;
  for (int k = 0, t; ok && (t = sc.tile(k)) >= 0; ++k) {
    const XTile ti = decode(P, sc, t, rank);
    const XJob& g = P.job[ti.p];
    const int n0 = ti.n0 + rank * (g.tn / 2) + g.b_n0;
    const uint32_t bytes = 2 * (kABytes + g.tn * 64);   // both CTAs' A rows and halves of B
    for (int kb = ti.kb0; kb < ti.kb1; ++kb, ++it) {
      const int s = it % kStages;
      if (!wait_bar_cluster(&empty[s], ((it / kStages) & 1) ^ 1, wc)) { ok = false; break; }
      const uint32_t fbar = mapa_shared(smem_u32(&full[s]), 0);
      uint8_t* sA = stages + s * kStageBytes;
      const int k0 = kb * kBK;
      if (part == 0) {
        if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
        if (g.a_mn) {
          tma_load_2d_pair(sA, &g.tmA, ti.m0, k0, fbar);
          tma_load_2d_pair(sA + kAtomBytes, &g.tmA, ti.m0 + 64, k0, fbar);
        } else {
          tma_load_2d_pair(sA, &g.tmA, k0, ti.m0, fbar);
        }
      } else {
        uint8_t* sB = sA + kABytes;
        if (P.split && ti.kind == XK_DW) {       // X's rows for either part of dz
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tma_load_2d_pair(sB + i * (kAtomBytes / 2), &g.tmB, n0, 0, fbar);
            tma_load_2d_pair(sB + kAtomBytes + i * (kAtomBytes / 2), &g.tmB, n0 + 64, 0, fbar);
          }
        } else if (g.b_mn) {
          tma_load_2d_pair(sB, &g.tmB, n0, k0 + g.b_k0, fbar);
          tma_load_2d_pair(sB + kAtomBytes, &g.tmB, n0 + 64, k0 + g.b_k0, fbar);
        } else {
          tma_load_2d_pair(sB, &g.tmB, k0 + g.b_k0, n0, fbar);
        }
      }
    }
  }
  // the latest use of every stage has landed before the CTA leaves
  if (rank == 0 && part == 0) {
    const int n = it < kStages ? it : kStages;
    for (int q = 1; q <= n; ++q) {
      const int u = it - q;
      wait_bar_drain(&full[u % kStages], (u / kStages) & 1, wc.limit_ns);
    }
  }
}

// One thread of the leader CTA issues every MMA of the pair.  A tile goes
// through one accumulator, or (forward) one after another per segment of K;
// every tile has K blocks.
template <bool BWD>
__device__ void mma_role(const XParams& P, const Schedule& sc, uint8_t* stages, uint64_t* full,
                         uint64_t* empty, uint64_t* tfull, uint64_t* tempty, uint64_t* drain,
                         uint32_t tmem_base, const WaitCtl& wc) {
  int acc = 0, s = 0;
  uint32_t ph = 0, soff = 0;
  const uint32_t sbase = smem_u32(stages);
  bool ok = true;
  for (int k = 0, t; ok && (t = sc.tile(k)) >= 0; ++k) {
    const XTile ti = decode(P, sc, t, 0);
    const XJob& g = P.job[ti.p];
    const uint32_t a_mn = g.a_mn ? 1u : 0u, b_mn = g.b_mn ? 1u : 0u;
    // D fp32, A and B bf16, their majors, N, M = 256
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (a_mn << 15) | (b_mn << 16) |
                           ((uint32_t)(g.tn >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
    const uint64_t a0 = smem_desc_sw128(sbase, a_mn ? kAtomBytes : 16, 1024);
    const uint64_t b0 = smem_desc_sw128(sbase + kABytes, b_mn ? kAtomBytes : 16, 1024);
    // an MMA's K step: 16 rows of an MN-major block, or 32 bytes of a row
    const uint32_t ak = a_mn ? (16 * 128) >> 4 : 2, bk = b_mn ? (16 * 128) >> 4 : 2;
    for (int kb = ti.kb0; kb < ti.kb1;) {
      const int buf = acc & 1;
      if (!wait_bar_cluster(&tempty[buf], ((acc >> 1) & 1) ^ 1, wc)) { ok = false; break; }
      tc_fence_after();
      const uint32_t d = tmem_base + buf * kTile;
      const int first = kb, end = BWD ? ti.kb1 : min(kb + P.segment, ti.kb1);
      for (; kb < end; ++kb) {
        if (!wait_bar_cluster(&full[s], ph, wc)) { ok = false; break; }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_pair(d, a0 + soff + kk * ak, b0 + soff + kk * bk, idesc, kb != first || kk != 0);
        tc_commit_pair(&empty[s], 3);
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
          soff = 0;
        } else {
          soff += kStageBytes >> 4;
        }
      }
      if (!ok) break;
      tc_commit_pair(&tfull[buf], 3);
      ++acc;
    }
  }
  tc_commit_pair(drain, 1);
  wait_bar_drain(drain, 0, wc.limit_ns);
}

// The gradient that reaches the losses: one factor for all rows (SUM, MEAN)
// multiplies dX and dW in fp32, so dz = exp(z - lse) - onehot is rounded to
// bf16 without it (at a target that is not predicted dz is about -1, which
// bf16 holds; a factor such as 1/1000 would put the same rounding error into
// every such row).  A factor per row (NONE) goes into dz.
__device__ __forceinline__ float common_scale(const float* dloss, const float* total, int reduction) {
  if (reduction == MOE_REDUCE_NONE) return 1.f;
  if (reduction == MOE_REDUCE_SUM) return dloss[0];
  return dloss[0] / fmaxf(total[2], 1.f);   // total[2]: rows that count
}

// Load 16 consecutive fp32 columns of the warp's 32 TMEM lanes (half of
// tmem_ld32, where a row's 128 sums leave few registers).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

struct BulkCopies {
  template <int N>
  __device__ __forceinline__ void wait_read() { bulk_wait_read<N>(); }
  __device__ __forceinline__ void commit() { bulk_commit(); }
};

template <bool BWD>
__device__ void epilogue_role(const XParams& P, const Schedule& sc, int rank, uint64_t* tfull,
                              uint64_t* tempty, uint32_t tmem_base, uint8_t* stg, const WaitCtl& wc) {
  const int ew = (threadIdx.x >> 5) - 2;
  const int q = (threadIdx.x >> 5) & 3;          // TMEM lane quarter of this warp
  const int half = ew >> 2;                      // which half of the tile's columns
  const int lane = threadIdx.x & 31;
  uint8_t* sb0 = stg + ew * 4096;
  uint8_t* sb1 = sb0 + 2048;
  const uint32_t te0 = mapa_shared(smem_u32(&tempty[0]), 0);
  const uint32_t te1 = mapa_shared(smem_u32(&tempty[1]), 0);
  StagingTurns<BulkCopies> turns;                // (lane 0's)
  // 64 columns of bf16 results as two boxes, a staging buffer each; columns at
  // or past `cols` are left out.  A buffer is written again once its own last
  // store has been read, while the other's may still be on its way.
  auto store_box = [&](const CUtensorMap* m, uint8_t* buf, const float (&v)[32], int x, int y) {
    if (lane == 0) turns.before_box();
    __syncwarp();
    stage_bf16_row(buf, lane, v);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(m, buf, x, y);
      turns.after_box();
    }
  };
  auto store_boxes = [&](const CUtensorMap* m, const float (&a)[32], const float (&b)[32], int x, int y,
                         int cols) {
    if (x < cols) store_box(m, sb0, a, x, y);
    else if (lane == 0) turns.after_box();
    if (x + 32 < cols) store_box(m, sb1, b, x + 32, y);
    else if (lane == 0) turns.after_box();
  };
  const float gs = BWD ? common_scale(P.dloss, P.total, P.reduction) : 1.f;
  int acc = 0;                                   // accumulators taken so far
  // waits for the next accumulator, and gives it back
  auto take = [&]() {
    const bool got = wait_bar_cluster(&tfull[acc & 1], (acc >> 1) & 1, wc);
    if (!__all_sync(0xffffffffu, got)) return false;
    tc_fence_after();
    return true;
  };
  auto give = [&]() {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(acc & 1 ? te1 : te0);
    ++acc;
  };
  for (int k = 0, t; (t = sc.tile(k)) >= 0; ++k) {
    const XTile ti = decode(P, sc, t, rank);
    const XJob& g = P.job[ti.p];
    const int y0 = ti.m0 + q * 32;               // first row of this warp
    const int row = y0 + lane;
    const int cw = g.tn / 2, c0 = half * cw;     // this warp's columns
    const bool rows = ti.kind != XK_DW;          // output rows are tokens
    const bool live = !rows || row < P.T;
    int tgt = -1;
    float lse2 = 0.f, scale = 0.f;
    if (ti.kind <= XK_DZ && live) {
      tgt = target_of(P.targets, P.index64, P.ignore_index, P.V, row);
      if (BWD && tgt == -2 && ti.n0 == 0) report(P.status, MOE_ERR_BAD_INDEX);
      if (BWD && tgt >= 0) {
        lse2 = P.lse[row] * kLog2e;
        scale = P.reduction == MOE_REDUCE_NONE ? P.dloss[row] : 1.f;
      }
    }
    const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16) + c0;
    if constexpr (!BWD) {
      const int v0 = ti.n0 + c0;                 // first vocabulary entry of this warp
      float z[4][32] = {};                       // the row's logits (cw of them)
      bool got = true;
      for (int kb = ti.kb0; kb < ti.kb1; kb += P.segment) {
        got = take();
        if (!got) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (16 * c >= cw) continue;
          float v[16];
          tmem_ld16(lanes + (acc & 1) * kTile + 16 * c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) z[c >> 1][16 * (c & 1) + i] += v[i];
        }
        give();
      }
      if (!got) break;
      float m = -INFINITY, s = 0.f;              // of the logits times log2(e)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (32 * c >= cw) continue;
        if (v0 + 32 * c + 32 > P.V) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (v0 + 32 * c + i >= P.V) z[c][i] = -INFINITY;
        }
        const int rel = tgt - (v0 + 32 * c);
        if (__any_sync(0xffffffffu, tgt >= 0 && rel >= 0 && rel < 32)) {
          float zt = 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i) zt = rel == i ? z[c][i] : zt;
          if (tgt >= 0 && rel >= 0 && rel < 32) P.zt[row] = zt * kLog2e;
        }
        float cm = z[c][0];
#pragma unroll
        for (int i = 1; i < 32; ++i) cm = fmaxf(cm, z[c][i]);
        const float mn = fmaxf(m, cm * kLog2e);
        const float ref = mn == -INFINITY ? 0.f : mn;   // nothing finite so far: every term is 0
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          a += ex2(fmaf(z[c][i], kLog2e, -ref));
          b += ex2(fmaf(z[c][i + 1], kLog2e, -ref));
        }
        s = s * ex2(m - ref) + (a + b);
        m = mn;
      }
      if (live) P.part[(size_t)(2 * ti.ntile + half) * P.T + row] = make_float2(m, s);
      continue;
    }
    if (!take()) break;
    const uint32_t taddr = lanes + (acc & 1) * kTile;
    if (ti.kind == XK_DZ) {
      const int v0 = g.b_n0 + ti.n0 + c0;
#pragma unroll 1
      for (int c = 0; c < cw; c += 64) {         // (96 columns: the second box of the last turn is left out)
        float a[32], b[32];
        const bool two = c + 32 < cw;
        tmem_ld32x2(taddr + c, taddr + (two ? c + 32 : c), a, b);
        const int rel = tgt - (v0 + c);
        const bool here = __any_sync(0xffffffffu, tgt >= 0 && rel >= 0 && rel < 64);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          a[i] = ex2(fmaf(a[i], kLog2e, -lse2));
          b[i] = ex2(fmaf(b[i], kLog2e, -lse2));
        }
        if (here) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            a[i] -= rel == i ? 1.f : 0.f;
            b[i] -= rel == i + 32 ? 1.f : 0.f;
          }
        }
        // an ignored row is exactly zero, whatever its logits; so are the
        // columns past the vocabulary that pad the last piece
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          a[i] = tgt >= 0 ? a[i] * scale : 0.f;
          b[i] = tgt >= 0 ? b[i] * scale : 0.f;
        }
        if (v0 + c + 64 > P.V) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (v0 + c + i >= P.V) a[i] = 0.f;
            if (v0 + c + 32 + i >= P.V) b[i] = 0.f;
          }
        }
        const int x = ti.n0 + c0 + c, end = two ? P.zcols : min(P.zcols, x + 32);
        if (y0 < P.T) store_boxes(&g.tmO, a, b, x, y0, end);
        if (y0 < P.T && P.split) {               // (y0 is 0) what that rounding left, 32 rows on
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            a[i] -= __bfloat162float(__float2bfloat16_rn(a[i]));
            b[i] -= __bfloat162float(__float2bfloat16_rn(b[i]));
          }
          store_boxes(&g.tmO, a, b, x, kSplitRows, end);
        }
      }
    } else if (ti.kind == XK_DX && P.last) {     // the sums of the pieces before + this one, to bf16
      const float* sums = P.acc + ((size_t)ti.slice * P.T + (live ? row : 0)) * P.Hp + ti.n0 + c0;
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        float a[32], b[32], u[32];
        tmem_ld32x2(taddr + c, taddr + c + 32, a, b);
        if (P.add && live) {
          load32<float>(sums + c, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) a[i] += u[i];
          load32<float>(sums + c + 32, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) b[i] += u[i];
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          a[i] *= gs;
          b[i] *= gs;
        }
        if (y0 < P.T) store_boxes(&g.tmO, a, b, ti.n0 + c0 + c, y0, P.H);
      }
    } else if (ti.kind == XK_DX) {               // fp32 sums, written or added to by bulk copies
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        float v[32];
        tmem_ld32(taddr + c, v);
        if (y0 >= P.rows) continue;
        if (lane == 0) turns.before_both();
        __syncwarp();
        stage_f32_row(sb0, lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (P.add) tma_add_3d(&g.tmO, sb0, ti.n0 + c0 + c, y0, ti.slice);
          else tma_store_3d(&g.tmO, sb0, ti.n0 + c0 + c, y0, ti.slice);
          turns.after_both();
        }
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        float a[32], b[32];
        tmem_ld32x2(taddr + c, taddr + c + 32, a, b);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          a[i] *= gs;
          b[i] *= gs;
        }
        if (g.out_m0 + y0 < P.V) store_boxes(&g.tmO, a, b, ti.n0 + c0 + c, g.out_m0 + y0, P.H);
      }
    }
    give();
  }
  if (lane == 0) bulk_wait_all();
  __syncwarp();
}

template <bool BWD>
__global__ void __launch_bounds__(kThreads, 1) xent_gemm_kernel(const __grid_constant__ XParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* stages = smem;
  uint8_t* stg = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + kStgBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int rank = (int)cluster_ctarank();
  let_next_start();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    for (int p = 0; p < P.njob; ++p) {
      tma_prefetch_desc(&P.job[p].tmA);
      tma_prefetch_desc(&P.job[p].tmB);
    }
  }
  if (warp == 1) tmem_alloc_pair(tmem_holder, 2 * kTile);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                            // the peer's barriers exist
  tc_fence_after();
  wait_for_previous();
  if (!BWD && blockIdx.x == 0 && threadIdx.x == 0) *P.ticket = 0;   // of the join kernel
  const uint32_t tmem_base = *tmem_holder;
  const Schedule sc(P);
  const WaitCtl wc{abort_flag, P.status, P.wait_ns};
  if (warp == 0) {
    if ((threadIdx.x & 31) == 0) load_role(P, sc, rank, stages, full, empty, wc, 0);
    __syncwarp();
  } else if (warp == 1) {
    if ((threadIdx.x & 31) == 0 && rank == 0)
      mma_role<BWD>(P, sc, stages, full, empty, tfull, tempty, drain, tmem_base, wc);
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    epilogue_role<BWD>(P, sc, rank, tfull, tempty, tmem_base, stg, wc);
  } else {
    if ((threadIdx.x & 31) == 0) load_role(P, sc, rank, stages, full, empty, wc, 1);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // after an abort, copies that either CTA issued may still be on their way
  // to the other: they land within microseconds
  if (threadIdx.x == 0 && *abort_flag) {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 200000) __nanosleep(1000);
  }
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 2 * kTile);
}

// Joins the pieces of each row (32 rows per block, a warp per slice of the
// pieces with a lane per row, so reads are coalesced; then a tree over the
// warps), and sums the losses up: each block its rows, the last block to
// finish all blocks' sums, in their order.
struct BlockSum {
  double sum;
  int count, pad;
};

__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float mn = fmaxf(m, m2);
  const float ref = mn == -INFINITY ? 0.f : mn;
  s = s * ex2(m - ref) + s2 * ex2(m2 - ref);
  m = mn;
}

__device__ __forceinline__ void warp_sum(double& s, int& n) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
}

__global__ void __launch_bounds__(1024) xent_join_kernel(const float2* part, int np, const float* zt,
                                                         const void* targets, int index64, int ignore,
                                                         int T, int V, float* loss, float* lse,
                                                         BlockSum* sums, unsigned* ticket,
                                                         float* total, int32_t* status) {
  __shared__ float2 sm[32][33];
  __shared__ double ss[32];
  __shared__ int sc[32];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane, r = blockIdx.x * 32 + w;
  float m = -INFINITY, s = 0.f;
  let_next_start();
  wait_for_previous();
  // what the row's last step needs, asked for early (z is read for a valid target only)
  const int t = r < T ? target_of(targets, index64, ignore, V, r) : -1;
  const float z = t >= 0 ? zt[r] : 0.f;
  if (row < T)
    for (int i = w; i < np; i += 128) {          // four pieces at a time
      float2 p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        p[k] = i + 32 * k < np ? part[(size_t)(i + 32 * k) * T + row] : make_float2(-INFINITY, 0.f);
      const float mn = fmaxf(m, fmaxf(fmaxf(p[0].x, p[1].x), fmaxf(p[2].x, p[3].x)));
      const float ref = mn == -INFINITY ? 0.f : mn;
      s *= ex2(m - ref);
#pragma unroll
      for (int k = 0; k < 4; ++k) s += p[k].y * ex2(p[k].x - ref);
      m = mn;
    }
  sm[lane][w] = make_float2(m, s);
  __syncthreads();
  // warp w joins the 32 slices of row w
  const float2 mine = sm[w][lane];
  m = mine.x;
  s = mine.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, m2, s2);
  }
  if (lane == 0) {
    double mine_loss = 0.0;
    int counts = 0;
    if (r < T) {
      // (the loss from differences of logits, not of lse: a small one keeps its digits)
      constexpr float kLn2 = 0.6931471805599453f;
      const float lg = log2f(s), l = (m + lg) * kLn2;
      if (t == -2) report(status, MOE_ERR_BAD_INDEX);
      counts = t >= 0;
      const float v = counts ? ((m - z) + lg) * kLn2 : 0.f;
      lse[r] = l;
      loss[r] = v;
      mine_loss = v;
    }
    ss[w] = mine_loss;
    sc[w] = counts;
  }
  __syncthreads();
  if (gridDim.x > 1) {
    if (w == 0) {
      double a = ss[lane];
      int n = sc[lane];
      warp_sum(a, n);
      if (lane == 0) {
        sums[blockIdx.x] = BlockSum{a, n, 0};
        __threadfence();
        last = atomicAdd(ticket, 1u) == gridDim.x - 1;
      }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double a = 0.0;
    int n = 0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 1024) {
      a += __ldcg(&sums[i].sum);
      n += __ldcg(&sums[i].count);
    }
    warp_sum(a, n);
    if (lane == 0) {
      ss[w] = a;
      sc[w] = n;
    }
    __syncthreads();
  }
  if (w) return;
  double a = ss[lane];
  int n = sc[lane];
  warp_sum(a, n);
  if (lane == 0) {
    total[0] = (float)a;
    total[1] = n ? (float)(a / n) : 0.f;
    total[2] = (float)n;
  }
}

// ------------------------------------------------------------ few tokens
// The forward for at most 16 tokens (scoring while generating): the bound is
// reading W once, and a 256-row MMA tile would be nearly empty.  A warp takes
// 16 vocabulary rows at a time straight from memory into the fragments of
// m16n8k16 products (A: the rows, B: the tokens, from shared memory).  K may be
// taken in any order as long as both operands agree, so a lane's four K
// positions of two consecutive products are eight adjacent columns: one
// 16-byte load per row.  Every lane keeps a running maximum and sum of its
// tokens over all rows it sees; lanes, warps and blocks are joined at the end.
// Measured: V = 131072, H = 4096, 8 tokens: 161 us with the join (6.7 TB/s);
// V = 32000, H = 2048, 7 tokens: 26.5 us, where the 256-row tiles take 49.
// Loads four chunks ahead are 4% slower, more and smaller blocks 10% and more.
constexpr int kFewWarps = 8, kFewPerSm = 2, kFewAhead = 8;

struct FewArgs {
  const __nv_bfloat16* X;
  const __nv_bfloat16* W;
  const void* targets;
  float2* part;
  float* zt;
  unsigned* ticket;
  int64_t ld_x, ld_w;
  int T, H, V, index64, ignore, pitch;   // pitch: bytes of a token's row in shared memory
};

__device__ __forceinline__ uint4 load_stream16(const void* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NB>   // blocks of 8 tokens
__global__ void __launch_bounds__(32 * kFewWarps, kFewPerSm) xent_few_kernel(const FewArgs a) {
  extern __shared__ __align__(16) uint8_t xs[];          // [8 NB][pitch]
  __shared__ float2 sm[kFewWarps][8 * NB];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  let_next_start();
  wait_for_previous();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  const int words = a.pitch / 16;
  for (int i = threadIdx.x; i < 8 * NB * words; i += 32 * kFewWarps) {
    const int n = i / words, c = (i - n * words) * 8;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (n < a.T && c < a.H) u = *reinterpret_cast<const uint4*>(a.X + n * a.ld_x + c);
    *reinterpret_cast<uint4*>(xs + n * a.pitch + c * 2) = u;
  }
  int tgt[2 * NB];
  float m[2 * NB], s[2 * NB];
#pragma unroll
  for (int j = 0; j < 2 * NB; ++j) {
    const int n = (j >> 1) * 8 + 2 * t + (j & 1);
    tgt[j] = n < a.T ? target_of(a.targets, a.index64, a.ignore, a.V, n) : -1;
    m[j] = -INFINITY;
    s[j] = 0.f;
  }
  __syncthreads();
  const int tasks = (a.V + 15) / 16, chunks = (a.H + 31) / 32;
  const uint8_t* xl = xs + g * a.pitch + t * 16;          // this lane's part of B
  // consecutive tasks go to different blocks, so that the last, partial round
  // is spread over all SMs
  for (int task = w * gridDim.x + blockIdx.x; task < tasks; task += kFewWarps * gridDim.x) {
    const int r0 = task * 16 + g, r1 = r0 + 8;
    const __nv_bfloat16* p0 = a.W + (int64_t)r0 * a.ld_w + t * 8;
    const __nv_bfloat16* p1 = a.W + (int64_t)r1 * a.ld_w + t * 8;
    float c[NB][4] = {}, z[NB][4] = {};
    uint4 u0[kFewAhead], u1[kFewAhead];
    auto load = [&](int q, uint4& x, uint4& y) {
      const bool in = q * 32 + t * 8 < a.H;
      x = in && r0 < a.V ? load_stream16(p0 + q * 32) : make_uint4(0, 0, 0, 0);
      y = in && r1 < a.V ? load_stream16(p1 + q * 32) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < kFewAhead; ++i) load(i, u0[i], u1[i]);
    for (int q = 0; q < chunks; q += kFewAhead) {
#pragma unroll
      for (int i = 0; i < kFewAhead; ++i) {
        const uint4 x = u0[i], y = u1[i];
        load(q + i + kFewAhead, u0[i], u1[i]);
        if (q + i < chunks) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint4 v = *reinterpret_cast<const uint4*>(xl + b * 8 * a.pitch + (q + i) * 64);
            mma_16x8x16(c[b], x.x, y.x, x.y, y.y, v.x, v.y);
            mma_16x8x16(c[b], x.z, y.z, x.w, y.w, v.z, v.w);
          }
        }
      }
      // segments of 256 columns, for the reason given at the top (here they cost nothing)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[b][i] += c[b][i];
          c[b][i] = 0.f;
        }
    }
    // z[b][0], z[b][1]: row r0, tokens 8 b + 2 t, + 1;  z[b][2], z[b][3]: row r1
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) {
      const float z0 = z[j >> 1][j & 1] * kLog2e, z1 = z[j >> 1][2 + (j & 1)] * kLog2e;
      const int n = (j >> 1) * 8 + 2 * t + (j & 1);
      if (tgt[j] >= 0 && tgt[j] == r0) a.zt[n] = z0;
      if (tgt[j] >= 0 && tgt[j] == r1) a.zt[n] = z1;
      if (r0 < a.V) join(m[j], s[j], z0, 1.f);
      if (r1 < a.V) join(m[j], s[j], z1, 1.f);
    }
  }
#pragma unroll
  for (int j = 0; j < 2 * NB; ++j) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[j], o), s2 = __shfl_xor_sync(0xffffffffu, s[j], o);
      join(m[j], s[j], m2, s2);
    }
    if (g == 0) sm[w][(j >> 1) * 8 + 2 * t + (j & 1)] = make_float2(m[j], s[j]);
  }
  __syncthreads();
  const int n = threadIdx.x;
  if (n < a.T) {
    float2 v = sm[0][n];
#pragma unroll
    for (int i = 1; i < kFewWarps; ++i) join(v.x, v.y, sm[i][n].x, sm[i][n].y);
    a.part[(size_t)blockIdx.x * a.T + n] = v;
  }
}

// dX from the slices' fp32 sums (H a multiple of 8).
__global__ void __launch_bounds__(256) xent_dx_kernel(const float* acc, int ks, int rows, int parts, int T, int H, int Hp,
                                                      const float* dloss, const float* total,
                                                      int reduction, __nv_bfloat16* dX) {
  let_next_start();
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = H / 8;
  if (i >= (int64_t)T * per) return;
  const int64_t row = i / per;
  const int c = (int)(i - row * per) * 8;
  float v[8] = {};
  const float* p = acc + (size_t)row * Hp + c;
  const size_t step = (size_t)rows * Hp, half = (size_t)kSplitRows * Hp;
#pragma unroll 8
  for (int k = 0; k < ks; ++k, p += step) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    if (parts > 1) {                             // the second part of a split dz
      const float4 e = *reinterpret_cast<const float4*>(p + half), f = *reinterpret_cast<const float4*>(p + half + 4);
      v[0] += e.x; v[1] += e.y; v[2] += e.z; v[3] += e.w;
      v[4] += f.x; v[5] += f.y; v[6] += f.z; v[7] += f.w;
    }
  }
  const float gs = common_scale(dloss, total, reduction);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= gs;
  *reinterpret_cast<uint4*>(dX + row * H + c) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                 pack_bf16(v[6], v[7]));
}

// ------------------------------------------------------------------ host
int up(int64_t a, int b) { return xent_up(a, b); }
size_t align256(size_t x) { return xent_align(x); }

// m-tiles that keep their rows of A in L2 (48 MB) through one sweep over N.
int group_for(int64_t row_bytes) {
  const int64_t g = (48LL << 20) / (kTile * row_bytes);
  return g < 1 ? 1 : (int)(g < 4096 ? g : 4096);
}

template <bool BWD>
cudaError_t launch(const XParams& P, cudaStream_t s) {
  auto kern = xent_gemm_kernel<BWD>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  static CtxCache<int> resident;   // pairs that run at once, per context
  int pairs = 0;
  cudaError_t e = resident.get(&pairs, [&](int* v) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (r != cudaSuccess) return r;
    cudaLaunchConfig_t c = cfg;
    c.numAttrs = 1;
    c.gridDim = dim3(2 * (sm_count() / 2), 1, 1);
    int n = 0;
    r = cudaOccupancyMaxActiveClusters(&n, kern, &c);
    if (r == cudaSuccess && n < 1) r = cudaErrorInvalidConfiguration;
    *v = n;
    return r;
  });
  if (e != cudaSuccess) return e;
  int64_t tiles = 0;
  for (int p = 0; p < P.njob; ++p) tiles += (int64_t)P.job[p].mt * P.job[p].nt * P.job[p].ks;
  if (tiles < pairs) pairs = (int)tiles;
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, P);
}

struct FwdWs {
  size_t part, zt, sums, ticket, total;
};
// The size does not depend on the GPU (it is asked for without one): room for
// the pieces of either kernel, at either tile width.
FwdWs fwd_ws(const XentDesc& d) {
  FwdWs w;
  int64_t np = 2 * (int64_t)up(d.V, 192);
  if (d.T <= kFewTokens && np < kFewMaxBlocks) np = kFewMaxBlocks;
  size_t o = 0;
  w.part = o; o += align256((size_t)np * d.T * sizeof(float2));
  w.zt = o; o += align256((size_t)d.T * sizeof(float));
  w.sums = o; o += align256((size_t)up(d.T, 32) * sizeof(BlockSum));
  w.ticket = o; o += 256;
  w.total = o;
  return w;
}

// Bytes of a token's row in the shared memory of the kernel for few tokens:
// whole 32-column chunks, and 64 bytes more than a multiple of 128, so that
// the eight lanes of a quarter-warp read different banks.
int few_pitch(int H) { return (H * 2 + 127) / 128 * 128 + 64; }
bool few_tokens(const XentDesc& d) {
  return d.T <= kFewTokens && (int64_t)(d.T <= 8 ? 8 : 16) * few_pitch(d.H) <= 110 * 1024;
}

template <int NB>
cudaError_t run_few(const FewArgs& a, int* blocks, cudaStream_t s) {
  static CtxCache<int> opt_in;
  int ok = 0;
  const cudaError_t e = opt_in.get(&ok, [](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(xent_few_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, 110 * 1024);
  });
  if (e != cudaSuccess) return e;
  const int tasks = (a.V + 15) / 16;
  int n = kFewPerSm * sm_count();
  if (n > kFewMaxBlocks) n = kFewMaxBlocks;
  if (n > tasks) n = tasks;
  *blocks = n;
  return launch_overlapped(xent_few_kernel<NB>, n, 32 * kFewWarps, 8 * NB * a.pitch, s, a);
}

cudaError_t launch_few(const XentDesc& d, const void* X, const void* W, const void* targets, float2* part,
                       float* zt, unsigned* ticket, int* np, cudaStream_t s) {
  const FewArgs a{static_cast<const __nv_bfloat16*>(X), static_cast<const __nv_bfloat16*>(W), targets, part,
                  zt, ticket, d.ld_x, d.ld_w, d.T, d.H, d.V, d.index_type == MOE_INDEX_I64, d.ignore_index,
                  few_pitch(d.H)};
  return d.T <= 8 ? run_few<1>(a, np, s) : run_few<2>(a, np, s);
}

XParams params_of(const XentDesc& d, const void* targets, int32_t* status) {
  XParams P;
  memset(&P, 0, sizeof(P));
  P.T = d.T;
  P.H = d.H;
  P.V = d.V;
  P.targets = targets;
  P.index64 = d.index_type == MOE_INDEX_I64;
  P.ignore_index = d.ignore_index;
  P.status = status;
  P.wait_ns = d.wait_ns;
  return P;
}

// Width of the logit tiles: 256 columns, or 192 where that saves enough of the
// last, partly filled round of tiles over the SM pairs to make up for the
// operand bytes, a sixth more per product.  Measured, forward: T = 1001, H =
// 1032, V = 10007 (three rounds of either) 28.8 against 30.6 us; T = 1500, H =
// 2048, V = 30000 (no round saved) 141 against 117 us.
int tile_width(int T, int cols, int pairs) {
  const int64_t mt = up(T, kTile);
  const int64_t r256 = up(mt * up(cols, 256), pairs) * 256LL, r192 = up(mt * up(cols, 192), pairs) * 192LL;
  return r192 * 115 < r256 * 100 ? 192 : 256;
}

bool logits_job(XJob& g, const XentDesc& d, const void* X, const void* W, int v0, int cols) {
  g.tn = tile_width(d.T, cols, sm_count() / 2);
  g.mt = up(d.T, kTile);
  g.nt = up(cols, g.tn);
  g.ks = 1;
  g.kblocks = up(d.H, kBK);
  g.group = group_for(2 * (int64_t)d.H);
  g.b_n0 = v0;
  return make_tmap(&g.tmA, X, 2, d.T, d.H, kBK, 128, d.ld_x) &&
         make_tmap(&g.tmB, W, 2, d.V, d.H, kBK, g.tn / 2, d.ld_w);
}

}  // namespace

size_t xent_forward_bytes(const XentDesc& d) { return fwd_ws(d).total; }
size_t xent_backward_bytes(const XentDesc& d) { return xent_backward_plan(d.T, d.H, d.V).total; }

#define XENT_TRY(expr)                       \
  do {                                       \
    const cudaError_t e_ = (expr);           \
    if (e_ != cudaSuccess) return e_;        \
  } while (0)

cudaError_t launch_xent_forward(const XentDesc& d, const void* X, const void* W, const void* targets,
                                float* loss, float* lse, float* total, char* ws, int32_t* status,
                                cudaStream_t s, moe_status* st) {
  *st = MOE_OK;
  const FwdWs w = fwd_ws(d);
  const int i64 = d.index_type == MOE_INDEX_I64;
  if (d.T == 0) return cudaMemsetAsync(total, 0, 3 * sizeof(float), s);
  float2* part = reinterpret_cast<float2*>(ws + w.part);
  float* zt = reinterpret_cast<float*>(ws + w.zt);
  unsigned* ticket = reinterpret_cast<unsigned*>(ws + w.ticket);
  int np = 0;
  if (few_tokens(d)) {
    XENT_TRY(launch_few(d, X, W, targets, part, zt, ticket, &np, s));
  } else {
    XParams P = params_of(d, targets, status);
    P.part = part;
    P.zt = zt;
    // segments of like length: none at a tile's end that is too short for the epilogue
    const int kblocks = up(d.H, kBK);
    P.segment = up(kblocks, up(kblocks, kSegment));
    P.ticket = ticket;
    P.njob = 1;
    P.job[0].kind = XK_STATS;
    if (!logits_job(P.job[0], d, X, W, 0, d.V)) {
      *st = MOE_ERR_CUDA;
      return cudaSuccess;
    }
    np = 2 * P.job[0].nt;
    XENT_TRY(launch<false>(P, s));
  }
  return launch_overlapped(xent_join_kernel, up(d.T, 32), 1024, 0, s, (const float2*)part, np, (const float*)zt,
                      targets, i64, d.ignore_index, d.T, d.V, loss, lse,
                      reinterpret_cast<BlockSum*>(ws + w.sums), ticket, total, status);
}

cudaError_t launch_xent_backward(const XentDesc& d, const void* X, const void* W, const void* targets,
                                 const float* lse, const float* total, const float* dloss,
                                 int reduction, void* dX, void* dW, char* ws, int32_t* status,
                                 cudaStream_t s, moe_status* st) {
  *st = MOE_OK;
  if (d.T == 0)   // no token: dW is zero
    return dW ? cudaMemsetAsync(dW, 0, (size_t)d.V * d.H * 2, s) : cudaSuccess;
  if (!dX && !dW) return cudaSuccess;
  const XentBackwardPlan w = xent_backward_plan(d.T, d.H, d.V);
  void* dz = ws + w.dz;
  const bool split = d.T <= kSplitRows, join = w.slices > 1 || split;   // a last kernel adds dX's sums up
  for (int v0 = 0; v0 < d.V; v0 += w.piece) {
    const int cols = d.V - v0 < w.piece ? d.V - v0 : w.piece;
    const bool last = v0 + cols == d.V;
    // dz of the piece
    XParams P = params_of(d, targets, status);
    P.dloss = dloss;
    P.total = total;
    P.reduction = reduction;
    P.lse = lse;
    P.zcols = w.piece;
    P.split = split;
    P.rows = w.rows;
    P.njob = 1;
    P.job[0].kind = XK_DZ;
    bool ok = logits_job(P.job[0], d, X, W, v0, cols) &&
              make_tmap_out(&P.job[0].tmO, dz, w.rows, w.piece, w.piece);
    if (ok) XENT_TRY(launch<true>(P, s));
    // dX (+)= dz W[piece], dW[piece] = dz^T X
    XParams Q = params_of(d, targets, status);
    Q.dloss = dloss;
    Q.total = total;
    Q.reduction = reduction;
    Q.acc = reinterpret_cast<float*>(ws + w.acc);
    Q.Hp = w.Hp;
    Q.add = v0 > 0;
    Q.last = last && !join;
    Q.split = split;
    Q.rows = w.rows;
    if (ok && dX) {
      XJob& g = Q.job[Q.njob++];
      g.kind = XK_DX;
      g.b_mn = 1;
      g.tn = kTile;
      g.mt = up(d.T, kTile);
      g.nt = up(d.H, kTile);
      g.kblocks = up(cols, kBK);
      g.ks = xent_piece_slices(w, cols);
      g.group = 8;
      g.b_k0 = v0;
      ok = make_tmap(&g.tmA, dz, 2, w.rows, w.piece, kBK, 128, w.piece) &&
           make_tmap(&g.tmB, W, 2, d.V, d.H, 64, kBK, d.ld_w) &&
           (Q.last ? make_tmap_out(&g.tmO, dX, d.T, d.H)
                   : make_tmap_out_f32(&g.tmO, Q.acc, w.slices, w.rows, w.Hp));
    }
    if (ok && dW) {
      XJob& g = Q.job[Q.njob++];
      g.kind = XK_DW;
      g.a_mn = g.b_mn = 1;
      g.tn = kTile;
      g.mt = up(cols, kTile);
      g.nt = up(d.H, kTile);
      g.kblocks = up(w.rows, kBK);
      g.ks = 1;
      g.group = 8;
      g.out_m0 = v0;
      ok = make_tmap(&g.tmA, dz, 2, w.rows, w.piece, 64, kBK, w.piece) &&
           make_tmap(&g.tmB, X, 2, d.T, d.H, 64, split ? kSplitRows : kBK, d.ld_x) && make_tmap_out(&g.tmO, dW, d.V, d.H);
    }
    if (!ok) {
      *st = MOE_ERR_CUDA;
      return cudaSuccess;
    }
    if (Q.njob == 2) {
      const int w0 = up(Q.job[0].kblocks, Q.job[0].ks), w1 = Q.job[1].kblocks;
      Q.catch_up = (w0 + w1 / 2) / w1;
    }
    XENT_TRY(launch<true>(Q, s));
  }
  if (dX && join) {
    const int64_t n = (int64_t)d.T * (d.H / 8);
    return launch_overlapped(xent_dx_kernel, (unsigned)((n + 255) / 256), 256, 0, s,
                        reinterpret_cast<const float*>(ws + w.acc), w.slices, w.rows, split ? 2 : 1, d.T, d.H, w.Hp, dloss, total,
                        reduction, static_cast<__nv_bfloat16*>(dX));
  }
  return cudaSuccess;
}

}  // namespace moe
