// rows.cuh - rows of a [T, H] tensor held by groups of lanes: what the norms
// over the hidden axis share.
//
// A row is held by L lanes (a power of two up to 32, or whole warps), every
// lane keeping the same CPT columns of each row.  A lane's vectors of the next
// rows travel to its own slots of shared memory (asynchronous copies that only
// this lane reads, so no barrier orders them).  Rows need not start on 16-byte
// boundaries (odd widths or strides: SHIFT): lanes are then laid over the
// aligned vectors that contain the row, whose first element sits m elements
// into its vector.  m repeats with a period of at most 8 rows, and a group of
// lanes takes rows of one m only (its stride over the rows is a multiple of the
// period), so its columns stay the same.  The vectors at a row's ends hold
// elements of its neighbours too: those are masked after the copy, and the
// stores there go by elements.  L and CPT are compile-time numbers: a row's
// offsets are then part of the instructions.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace rows {

// ------------------------------------------------------------- elements
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float load_w1(const void* p, int type, int c, float fill) {
  if (!p) return fill;
  return type == MOE_TYPE_BF16 ? to_f(static_cast<const __nv_bfloat16*>(p)[c])
                               : static_cast<const float*>(p)[c];
}

// Two fp32 numbers worked on by one instruction.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(F2 p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum2(F2 p) {
  float a, b;
  split(p, a, b);
  return a + b;
}

// ------------------------------------------------------------ reductions
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = W >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The barrier of one group's lanes (whole warps).
template <int THREADS>
__device__ __forceinline__ void group_bar(int group) {
  __syncwarp();
  asm volatile("barrier.sync %0, %1;" ::"r"(1 + group), "n"(THREADS) : "memory");
}

// Sums of N values over the L lanes of a row, given to all of them.  Up to a
// warp the N trees run side by side.  Beyond that a warp reduces two values
// together (the first exchange leaves one of them to each half) and one
// barrier joins the row's warps.  `sm` (N floats per warp of the block) is
// not written again before another barrier of the same group.
template <int N, int L>
__device__ __forceinline__ void row_sums(float (&v)[N], int group, float* sm) {
  static_assert(N == 1 || N == 2, "values per lane");
  if constexpr (L <= 32) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<L>(v[i]);
  } else {
    constexpr int W = 32 / N, WARPS = L / 32;    // lanes that carry one value
    const int lane = threadIdx.x & 31;
    float x = v[0];
    if constexpr (N == 2) {
      const bool up = lane & 16;
      x = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    }
    x = lanes_sum<W>(x);
    if ((lane & (W - 1)) == 0) sm[(threadIdx.x >> 5) * N + lane / W] = x;
    group_bar<L>(group);
    // each half (N == 2) or the whole warp adds the warps' sums up, as often
    // as they fit into its lanes
    constexpr int P = WARPS > 16 ? 32 : WARPS > 8 ? 16 : WARPS > 4 ? 8 : WARPS > 2 ? 4 : 2;
    const int k = lane / W, w = lane & ((P < W ? P : W) - 1);
    const float* g = sm + group * WARPS * N;
    x = w < WARPS ? g[w * N + k] : 0.f;
    if constexpr (WARPS > W) x += g[(w + W) * N + k];
    x = lanes_sum<(P < W ? P : W)>(x);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = N == 1 ? x : __shfl_sync(0xffffffffu, x, i * W);
  }
}

// 1 / sqrt(v): the approximation and one Newton step (below one ulp of fp32).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  // (0 and infinity have their values already; the step would make them NaN)
  return v > 0.f && v <= 3.402823466e38f ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}

// The same within half an ulp: the step's residual 1 - v r r is exact to 2^-40.
__device__ __forceinline__ float inv_sqrt_exact(float v) {
  const float r = rsqrtf(v), t = v * r;
  const float e = fmaf(-fmaf(v, r, -t), r, fmaf(-t, r, 1.f));
  return v > 0.f && v <= 3.402823466e38f ? fmaf(0.5f * r, e, r) : r;
}

// ------------------------------------------------------------------ rows
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Elements of a 16-byte vector.
template <typename X>
constexpr int kVec = 16 / (int)sizeof(X);

// A lane's CPT columns of every row of its group: element i of its vector j is
// column first() + j L V + i.  A vector lies wholly (full) or, at a row's ends
// with SHIFT, partly inside the row, or past it.
template <typename X, int CPT, int L, bool SHIFT>
struct Lane {
  static constexpr int V = kVec<X>;
  int t, c0, left;                       // c0: first column; left: columns from there to the row's end
  bool ends;                             // a lane of this warp holds an end of the row (SHIFT)
  __device__ __forceinline__ Lane(int H, int m)
      : t(threadIdx.x % L), c0(t * V - (SHIFT ? m : 0)), left(H - c0), ends(false) {
    if constexpr (SHIFT) {
#pragma unroll
      for (int j = 0; j < CPT / V; ++j) ends = ends || (valid(j) && !full(j));
      ends = __any_sync(0xffffffffu, ends);
    }
  }
  __device__ __forceinline__ int first() const { return c0; }
  __device__ __forceinline__ bool valid(int j) const { return left > j * L * V; }
  __device__ __forceinline__ bool full(int j) const {
    return SHIFT ? c0 + j * L * V >= 0 && left >= (j * L + 1) * V : valid(j);
  }
  // element i of vector j is in the row (asked of partly filled vectors)
  __device__ __forceinline__ bool inside(int j, int i) const {
    return c0 + j * L * V + i >= 0 && left > j * L * V + i;
  }
};

// A row's first element's place in its 16-byte vector.
template <typename X>
__device__ __forceinline__ int shift_of(const X* p) {
  return (int)((uintptr_t)p & 15) / (int)sizeof(X);
}

template <typename X, int CPT, int L, bool SHIFT>
__device__ __forceinline__ void store_row(const Lane<X, CPT, L, SHIFT>& l, X* row, const F2 (&p)[CPT / 2]) {
  constexpr int V = kVec<X>;
  row += l.first();
#pragma unroll
  for (int j = 0; j < CPT / V; ++j) {
    float e[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) split(p[j * V / 2 + i], e[2 * i], e[2 * i + 1]);
    X* q = row + j * L * V;
    if (SHIFT && l.ends ? l.full(j) : l.valid(j)) {
      if constexpr (sizeof(X) == 2)
        *reinterpret_cast<uint4*>(q) = make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]),
                                                  pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7]));
      else
        *reinterpret_cast<float4*>(q) = make_float4(e[0], e[1], e[2], e[3]);
    } else if (SHIFT && l.ends && l.valid(j)) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (l.inside(j, i)) put(q + i, e[i]);
    }
  }
}

// A lane's weights, read once per block (0 past the row's end): in registers
// up to 16 columns, else in shared memory (each lane's own, 16 bytes apart).
template <typename X, int CPT, int L, bool SHIFT, int THREADS>
struct Weights {
  static constexpr int V = kVec<X>;
  static constexpr bool REGS = CPT <= 16;
  F2 r[REGS ? CPT / 2 : 1];
  float4* s;
  __device__ __forceinline__ void load(const Lane<X, CPT, L, SHIFT>& l, const void* p, int type, float fill,
                                       float4* smem) {
    s = smem + threadIdx.x;
    F2 v[CPT / 2];
#pragma unroll
    for (int j = 0; j < CPT / V; ++j) {
      float e[V] = {};
      const int c = l.first() + j * L * V;
      if (l.valid(j)) {
        if (!SHIFT && V == 8 && p && type == MOE_TYPE_BF16 && ((uintptr_t)p & 15) == 0) {
          const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + c);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < V; ++i) e[i] = i & 1 ? bf16_hi(w[(i / 2) & 3]) : bf16_lo(w[(i / 2) & 3]);
        } else if (!SHIFT && p && type == MOE_TYPE_F32 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
          for (int i = 0; i + 3 < V; i += 4) {
            const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + i);
            e[i] = u.x; e[i + 1] = u.y; e[i + 2] = u.z; e[i + 3] = u.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (!SHIFT || l.inside(j, i)) e[i] = load_w1(p, type, c + i, fill);
        }
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) v[j * V / 2 + i] = f2(e[2 * i], e[2 * i + 1]);
    }
    if constexpr (REGS) {
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i) r[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < CPT / 4; ++i) {
        float4 f;
        split(v[2 * i], f.x, f.y);
        split(v[2 * i + 1], f.z, f.w);
        s[i * THREADS] = f;
      }
    }
  }
  __device__ __forceinline__ void get(F2 (&v)[CPT / 2]) const {
    if constexpr (REGS) {
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i) v[i] = r[i];
    } else {
#pragma unroll
      for (int i = 0; i < CPT / 4; ++i) {
        const float4 f = s[i * THREADS];
        v[2 * i] = f2(f.x, f.y);
        v[2 * i + 1] = f2(f.z, f.w);
      }
    }
  }
};

// The rows of one tensor on their way to a lane: a ring of S rows in shared
// memory, `at` the lane's first slot.  What lies past the row's ends reads as
// zero.
template <typename X, int CPT, int L, bool SHIFT, int S, int THREADS>
struct Stream {
  static constexpr int V = kVec<X>, NL = CPT / V;
  static constexpr int RING = S * NL * THREADS * 16;    // bytes per block
  using Lane_ = Lane<X, CPT, L, SHIFT>;
  const X* q;            // this lane's part of the next row to fetch
  int64_t ld, step;      // elements from row to row, and between this group's rows
  uint8_t* at;
  __device__ __forceinline__ Stream(const Lane_& l, const void* base, int64_t ld_, uint32_t row, uint32_t stride,
                                    uint8_t* ring)
      : q(static_cast<const X*>(base) + row * ld_ + l.first()), ld(ld_), step(stride * ld_),
        at(ring + threadIdx.x * 16) {
#pragma unroll
    for (int j = 0; j < NL; ++j)
      if (!l.valid(j))
        for (int st = 0; st < S; ++st)
          *reinterpret_cast<uint4*>(at + (st * NL + j) * THREADS * 16) = make_uint4(0, 0, 0, 0);
  }
  // Starts the copies of `row` (the group's next one) into ring stage st.
  __device__ __forceinline__ void fetch(const Lane_& l, uint32_t row, uint32_t T, int st) {
    if (row < T) copy(l, row, T, st);
    q += step;
  }
  __device__ __forceinline__ void copy(const Lane_& l, uint32_t row, uint32_t T, int st) {
    uint8_t* d = at + st * (NL * THREADS * 16);
    if (!SHIFT || !l.ends) {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if (l.valid(j)) copy_async16(smem_u32(d + j * THREADS * 16), q + j * L * V);
      return;
    }
    // elements from the tensor's first to this lane's, and to the tensor's end
    const int64_t before = (int64_t)row * ld + l.first();
    const int64_t after = (int64_t)(T - 1 - row) * ld + l.left;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      if (!l.valid(j)) continue;
      if (before + j * L * V >= 0 && after >= (j * L + 1) * V) {
        copy_async16(smem_u32(d + j * THREADS * 16), q + j * L * V);
      } else {                                   // the vector sticks out of the tensor itself
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (l.inside(j, i)) reinterpret_cast<X*>(d + j * THREADS * 16)[i] = q[j * L * V + i];
      }
    }
  }
  __device__ __forceinline__ void take(const Lane_& l, F2 (&x)[CPT / 2], int st) const {
    uint32_t w[NL][4];
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const uint4 u = *reinterpret_cast<const uint4*>(at + (st * NL + j) * THREADS * 16);
      w[j][0] = u.x; w[j][1] = u.y; w[j][2] = u.z; w[j][3] = u.w;
    }
    if (SHIFT && l.ends) {                       // elements of the rows before and after this one
#pragma unroll
      for (int j = 0; j < NL; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (!l.inside(j, i))
            w[j][i * (int)sizeof(X) / 4] &= sizeof(X) == 4 ? 0u : i & 1 ? 0x0000ffffu : 0xffff0000u;
    }
#pragma unroll
    for (int j = 0; j < NL; ++j)
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        x[j * V / 2 + i] = sizeof(X) == 2
                               ? f2(bf16_lo(w[j][i]), bf16_hi(w[j][i]))
                               : f2(__uint_as_float(w[j][(2 * i) & 3]), __uint_as_float(w[j][(2 * i + 1) & 3]));
  }
};

// Rows that a block of about N threads works on side by side, and its threads.
template <int L, int N>
constexpr int kRows = L > N / 2 ? 1 : N / L;
template <int L, int N>
constexpr int kBlock = kRows<L, N>* L;
template <typename X, int V>
__device__ __forceinline__ void load_part(const X* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f(*p);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = sizeof(X) == 4 ? __uint_as_float(w[i & 3]) : i & 1 ? bf16_hi(w[(i / 2) & 3]) : bf16_lo(w[(i / 2) & 3]);
  }
}
template <typename X, int V>
__device__ __forceinline__ void store_part(X* p, const float (&v)[V]) {
  if constexpr (V == 1)
    put(p, v[0]);
  else if constexpr (sizeof(X) == 2)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Where the rows of a call's tensors start relative to 16-byte boundaries.
struct Offsets {
  bool vectors;   // all on boundaries, and rows are whole vectors
  bool same;      // at the same offset in every tensor, row by row
  int period;     // rows after which the offset repeats (1 .. 8)
};
inline Offsets offsets_of(const void* const* p, const int64_t* ld, int n, int es, int T, int H) {
  Offsets o{(int64_t)H * es % 16 == 0, true, 1};
  for (int i = 0; i < n; ++i) {
    o.vectors = o.vectors && ((uintptr_t)p[i] & 15) == 0 && (T <= 1 || ld[i] * es % 16 == 0);
    o.same = o.same && (((uintptr_t)p[i] ^ (uintptr_t)p[0]) & 15) == 0 &&
             (T <= 1 || (ld[i] - ld[0]) * es % 16 == 0);
  }
  if (T > 1)
    while (ld[0] * es * o.period % 16) o.period *= 2;
  return o;
}

// Launches one form: blocks that fill the GPU once, but no more than there
// are rows; where a group takes several rows, their distance is a multiple of
// `period`.
template <typename Args, typename K>
cudaError_t run(K kern, CtxCache<int>& cache, const Args& a, int rows, int threads, int smem, int period,
                int64_t max_blocks, int* blocks_out, cudaStream_t s) {
  int per_sm = 0;
  const cudaError_t e = cache.get(&per_sm, [&](int* v) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kern, threads, smem);
    return r == cudaSuccess && *v < 1 ? cudaErrorInvalidConfiguration : r;
  });
  if (e != cudaSuccess) return e;
  int64_t blocks = (int64_t)sm_count() * per_sm;
  const int64_t need = ((int64_t)a.T + rows - 1) / rows;
  if (blocks > max_blocks) blocks = max_blocks;
  if (blocks >= need) {
    blocks = need;                       // a row per group
  } else {
    int unit = 1;                        // blocks in which whole periods of rows fit
    while (unit * rows % period) ++unit;
    blocks = blocks > unit ? blocks / unit * unit : unit;
  }
  *blocks_out = (int)blocks;
  return launch_overlapped(kern, (unsigned)blocks, threads, smem, s, a);
}

}  // namespace rows
}  // namespace moe
