// norm.cu - layer normalisation over the hidden axis, forward and backward.
//
//   forward   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//             y = (x - mu) r gamma + beta
//   backward  h = (x - mu) r, g = gamma dy:
//             dx = r (g - mean(g) - h mean(g h)),
//             dgamma = sum over rows of dy h,  dbeta = sum over rows of dy
//
// Both directions are bound by HBM: the forward moves 2 and the backward 3
// elements per element of x.  A row is held by L lanes (a power of two up to
// 32, or whole warps), every lane keeping the same columns of each row, so a
// row is read once, its statistics are taken from registers (the variance
// from centred values, in a second sum: no cancellation), gamma and beta are
// loaded once per block and the backward's column sums stay in registers over
// all rows of a block.  All sums are fp32 trees in a fixed order; the results
// do not depend on timing.
//
// Blocks are persistent.  A lane's vectors of the next rows travel to its own
// slots of shared memory (asynchronous copies that only this lane reads, so no
// barrier orders them).  Rows need not start on 16-byte boundaries (odd widths
// or strides: SHIFT): lanes are then laid over the aligned vectors that
// contain the row, whose first element sits m elements into its vector.  m
// repeats with a period of at most 8 rows, and a group of lanes takes rows of
// one m only (its stride over the rows is a multiple of the period), so its
// columns stay the same.  The vectors at a row's ends hold elements of its
// neighbours too: those are masked after the copy, and the stores there go by
// elements.  L and the columns per lane are compile-time numbers:
// a row's offsets are then part of the instructions, which with the arithmetic
// in pairs (fp32x2) keeps a row's instructions below the time that HBM takes
// for it (they were the bound of a first version with both at run time).
// Columns past the row's end read as zero; a group past the last row works on
// what its slots hold and stores nothing.
//
// Measured (GB300, bf16, gamma and beta bf16):
//   16384 x 4096, from HBM: forward 42.5 us (6.3 TB/s), backward 67 us (6.0
//   TB/s) and 4 - 6 us for the column sums' last step;
//   4097 x 2049, from L2: forward 11.8, backward 18.4 us; 2056 columns, on
//   vectors, 7.8 and 15.8 us;  one row of 4096: 2.3 and 4.9 us.
// From L2 the bound is the issue rate (13 instructions per element forward),
// from HBM its bandwidth.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

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
// The backward of bf16 rows has larger blocks: their column sums are joined in
// shared memory before they go to memory (16384 x 4096: 2 us less; fp32 rows
// fill the ring with fewer in flight: 5003 x 1536 takes 17.0 us so, 15.3 with
// 256 threads).
constexpr int kFwdThreads = 256;
template <typename X>
constexpr int kBwdThreads = sizeof(X) == 2 ? 512 : 256;

// --------------------------------------------------------------- forward
struct FwdArgs {
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  int64_t ld_x, ld_y;
  int T, H, wtype;
  float eps;
};

template <typename X, bool SHIFT, int CPT, int L, int S>
__global__ void __launch_bounds__(kBlock<L, kFwdThreads>, CPT <= 16 ? 800 / kBlock<L, kFwdThreads> : 1)
    norm_fwd_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int TH = kBlock<L, kFwdThreads>, ROWS = kRows<L, kFwdThreads>, V = kVec<X>;
  using Str = Stream<X, CPT, L, SHIFT, S, TH>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float sm[2][TH / 32];
  let_next_start();
  const int group = threadIdx.x / L;
  const uint32_t T = a.T, stride = gridDim.x * ROWS;   // (T below 2^31: rows past it do not wrap)
  uint32_t row = blockIdx.x * ROWS + group;
  const Lane<X, CPT, L, SHIFT> lane(
      a.H, SHIFT ? shift_of(static_cast<const X*>(a.x) + (row < T ? row : 0) * a.ld_x) : 0);
  Str xs(lane, a.x, a.ld_x, row, stride, dyn);
  X* out = static_cast<X*>(a.y) + row * a.ld_y;
  const int64_t out_step = stride * a.ld_y;
  wait_for_previous();
#pragma unroll
  for (int st = 0; st < S - 1; ++st) {
    xs.fetch(lane, row + st * stride, T, st);
    copy_commit();
  }
  Weights<X, CPT, L, SHIFT, TH> gam, bet;
  float4* wsm = reinterpret_cast<float4*>(dyn + Str::RING);
  gam.load(lane, a.gamma, a.wtype, 1.f, wsm);
  bet.load(lane, a.beta, a.wtype, 0.f, wsm + CPT / 4 * TH);
  const float inv = 1.f / (float)a.H;
  int st = 0;
  for (uint32_t base = blockIdx.x * ROWS; base < T; base += stride, row += stride) {
    F2 x[CPT / 2];
    xs.fetch(lane, row + (S - 1) * stride, T, st == 0 ? S - 1 : st - 1);
    copy_commit();
    copy_wait<S - 1>();
    xs.take(lane, x, st);
    if (++st == S) st = 0;
    F2 acc = f2(0.f, 0.f), acc2 = acc;
#pragma unroll
    for (int i = 0; i < CPT / 2; i += 2) {
      acc = add2(acc, x[i]);
      acc2 = add2(acc2, x[i + 1]);
    }
    float s[1] = {sum2(add2(acc, acc2))}, q[1] = {0.f};
    row_sums<1, L>(s, group, sm[0]);
    const float mu = s[0] * inv;
    const F2 neg = f2(-mu, -mu);
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) x[i] = add2(x[i], neg);
    if (SHIFT && lane.ends) {            // the row's ends, by elements
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float d[2];
        split(x[i / 2], d[0], d[1]);
        q[0] += lane.inside(i / V, i % V) ? d[i & 1] * d[i & 1] : 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < CPT / V; ++j) {
        F2 v = mul2(x[j * V / 2], x[j * V / 2]);
#pragma unroll
        for (int i = 1; i < V / 2; ++i) v = fma2(x[j * V / 2 + i], x[j * V / 2 + i], v);
        q[0] += lane.valid(j) ? sum2(v) : 0.f;
      }
    }
    row_sums<1, L>(q, group, sm[1]);
    const float r = inv_sqrt(q[0] * inv + a.eps);
    F2 g[CPT / 2], b[CPT / 2];
    gam.get(g);
    bet.get(b);
    const F2 rr = f2(r, r);
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) x[i] = fma2(mul2(x[i], rr), g[i], b[i]);
    if (row < T) {
      store_row(lane, out, x);
      if (lane.t == 0) {
        if (a.mean) a.mean[row] = mu;
        if (a.rstd) a.rstd[row] = r;
      }
    }
    out += out_step;
  }
  copy_wait<0>();
}

// Rows that the kernel above does not take (too long, or x and y at different
// offsets from 16-byte boundaries): a block per row, three passes over it (the
// second and third find most of it in L1 or L2), by vectors where all rows
// start on 16-byte boundaries (V = kVec), else by elements (V = 1).  Measured,
// bf16: 4097 x 2048 with tensors at different offsets 45 us forward and 69
// backward (4097 x 2049 at one offset 13 and 20); 4000 x 20000 184 and 366 (47 and
// 71 from HBM).
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

template <typename X, int V>
__global__ void __launch_bounds__(1024) norm_fwd_rows_kernel(const FwdArgs a) {
  __shared__ float sm[2][32];
  let_next_start();
  wait_for_previous();
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  float s[1] = {0.f}, q[1] = {0.f};
#pragma unroll 8
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float v[V];
    load_part(x + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] += v[i];
  }
  row_sums<1, 1024>(s, 0, sm[0]);
  const float mu = s[0] / (float)a.H;
#pragma unroll 8
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float v[V];
    load_part(x + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) q[0] += (v[i] - mu) * (v[i] - mu);
  }
  row_sums<1, 1024>(q, 0, sm[1]);
  const float r = inv_sqrt(q[0] / (float)a.H + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  X* y = static_cast<X*>(a.y) + row * a.ld_y;
#pragma unroll 2
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float v[V];
    load_part(x + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = (v[i] - mu) * r * load_w1(a.gamma, a.wtype, c + i, 1.f) + load_w1(a.beta, a.wtype, c + i, 0.f);
    store_part(y + c, v);
  }
}

// -------------------------------------------------------------- backward
struct BwdArgs {
  const void* dy;
  const void* x;
  const void* gamma;
  const float* mean;
  const float* rstd;
  void* dx;
  float* partial;      // [blocks][2][H]: dgamma and dbeta sums of each block
  int64_t ld_dy, ld_x, ld_dx;
  int T, H, wtype;
};

// With h = x r + b, b = -mu r, both means of a row follow from two sums, and
//   dx = r g + x A + B,  A = -r r mean(g h),  B = -r mean(g) - b r mean(g h).
// (Three blocks per SM instead of two, with gamma in shared memory and the row
// read from the ring a second time, measured no faster: 79 against 76 us.)
// GRADS: with the column sums of dgamma and dbeta.
template <typename X, bool SHIFT, int CPT, int L, int S, bool GRADS>
__global__ void __launch_bounds__(kBlock<L, kBwdThreads<X>>, CPT <= 16 ? 512 / kBlock<L, kBwdThreads<X>> : 1)
    norm_bwd_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int TH = kBlock<L, kBwdThreads<X>>, ROWS = kRows<L, kBwdThreads<X>>, V = kVec<X>;
  using Str = Stream<X, CPT, L, SHIFT, S, TH>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float sm[2][TH / 16];
  let_next_start();
  const int group = threadIdx.x / L;
  const uint32_t T = a.T, stride = gridDim.x * ROWS;   // (T below 2^31: rows past it do not wrap)
  uint32_t row = blockIdx.x * ROWS + group;
  const Lane<X, CPT, L, SHIFT> lane(
      a.H, SHIFT ? shift_of(static_cast<const X*>(a.x) + (row < T ? row : 0) * a.ld_x) : 0);
  Str xs(lane, a.x, a.ld_x, row, stride, dyn), ds(lane, a.dy, a.ld_dy, row, stride, dyn + Str::RING);
  X* dx = static_cast<X*>(a.dx) + row * a.ld_dx;
  const int64_t dx_step = stride * a.ld_dx;
  wait_for_previous();
#pragma unroll
  for (int st = 0; st < S - 1; ++st) {
    xs.fetch(lane, row + st * stride, T, st);
    ds.fetch(lane, row + st * stride, T, st);
    copy_commit();
  }
  auto at = [&](uint32_t q) { return q < T ? q : T - 1; };
  float mu = a.mean[at(row)], r = a.rstd[at(row)];
  Weights<X, CPT, L, SHIFT, TH> gam;
  gam.load(lane, a.gamma, a.wtype, 1.f, reinterpret_cast<float4*>(dyn + 2 * Str::RING));
  F2 dg[CPT / 2], db[CPT / 2];
#pragma unroll
  for (int i = 0; i < CPT / 2; ++i) dg[i] = db[i] = f2(0.f, 0.f);
  const float inv = 1.f / (float)a.H;
  int st = 0, par = 0;
  for (uint32_t base = blockIdx.x * ROWS; base < T; base += stride, row += stride) {
    const float rc = r, bc = -mu * r;
    const bool live = row < T;
    mu = a.mean[at(row + stride)];
    r = a.rstd[at(row + stride)];
    const int to = st == 0 ? S - 1 : st - 1;
    xs.fetch(lane, row + (S - 1) * stride, T, to);
    ds.fetch(lane, row + (S - 1) * stride, T, to);
    copy_commit();
    copy_wait<S - 1>();
    const F2 rr = f2(rc, rc), bb = f2(bc, bc);
    F2 s1 = f2(0.f, 0.f), s2 = s1;
    F2 x[CPT / 2], d[CPT / 2], g[CPT / 2];
    xs.take(lane, x, st);
    ds.take(lane, d, st);
    if (++st == S) st = 0;
    gam.get(g);
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) {
      const F2 h = fma2(x[i], rr, bb);
      const F2 gy = mul2(d[i], g[i]);
      s1 = add2(s1, gy);
      s2 = fma2(gy, h, s2);
      if (GRADS && live) {
        dg[i] = fma2(d[i], h, dg[i]);
        db[i] = add2(db[i], d[i]);
      }
      d[i] = gy;
    }
    float s[2] = {sum2(s1), sum2(s2)};
    row_sums<2, L>(s, group, sm[par]);
    par ^= 1;
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    const float A = -rc * rc * c2, B = -rc * c1 - bc * rc * c2;
    const F2 AA = f2(A, A), BB = f2(B, B);
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) x[i] = fma2(d[i], rr, fma2(x[i], AA, BB));
    if (live) store_row(lane, dx, x);
    dx += dx_step;
  }
  copy_wait<0>();
  if (!GRADS || !a.partial) return;
  // the block's column sums, through shared memory: groups of one block are
  // added in order, and the stores are coalesced
  float* out = a.partial + (size_t)blockIdx.x * 2 * a.H;
  float* acc = reinterpret_cast<float*>(dyn) + (size_t)group * 2 * a.H;   // [ROWS][2][H]
  __syncthreads();                       // the ring is no longer read
#pragma unroll
  for (int i = 0; i < CPT / 2; ++i) {
    float gs[2], bs[2];
    split(dg[i], gs[0], gs[1]);
    split(db[i], bs[0], bs[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = (2 * i + k) / V, e = (2 * i + k) % V, c = lane.first() + j * L * V + e;
      if (!(SHIFT ? lane.inside(j, e) : lane.valid(j))) continue;
      acc[c] = gs[k];
      acc[a.H + c] = bs[k];
    }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(dyn);
  for (int c = threadIdx.x; c < 2 * a.H; c += TH) {
    float v = all[c];
#pragma unroll
    for (int g = 1; g < ROWS; ++g) v += all[(size_t)2 * g * a.H + c];
    out[c] = v;
  }
}

// dgamma and dbeta from the blocks' partial sums: 32 columns per block, 32
// slices of the partials, added as a fixed tree.
__global__ void __launch_bounds__(1024) norm_param_grad_kernel(const float* partial, int blocks, int H,
                                                               int wtype, void* dgamma, void* dbeta) {
  __shared__ float sm[32][33];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H)
#pragma unroll 8
    for (int b = w; b < blocks; b += 32) v += partial[((size_t)b * 2 + blockIdx.y) * H + c];
  sm[w][lane] = v;
  __syncthreads();
  const float s = lanes_sum<32>(sm[lane][w]);   // warp w sums column w of the tile
  const int cw = blockIdx.x * 32 + w;
  void* out = blockIdx.y ? dbeta : dgamma;
  if (lane == 0 && cw < H && out) {
    if (wtype == MOE_TYPE_BF16) static_cast<__nv_bfloat16*>(out)[cw] = __float2bfloat16_rn(s);
    else static_cast<float*>(out)[cw] = s;
  }
}

// Rows that the kernel above does not take: dx with a block per row (two
// passes); the column sums from a read of their own, a thread per column.
template <typename X, int V>
__global__ void __launch_bounds__(1024) norm_bwd_rows_kernel(const BwdArgs a) {
  __shared__ float sm[64];
  let_next_start();
  wait_for_previous();
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  const X* dy = static_cast<const X*>(a.dy) + row * a.ld_dy;
  const float mu = a.mean[row], r = a.rstd[row];
  float s[2] = {0.f, 0.f};
#pragma unroll 4
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float d[V], v[V];
    load_part(dy + c, d);
    load_part(x + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float gy = d[i] * load_w1(a.gamma, a.wtype, c + i, 1.f);
      s[0] += gy;
      s[1] += gy * ((v[i] - mu) * r);
    }
  }
  row_sums<2, 1024>(s, 0, sm);
  const float c1 = s[0] / (float)a.H, c2 = s[1] / (float)a.H;
  X* dx = static_cast<X*>(a.dx) + row * a.ld_dx;
#pragma unroll 2
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float d[V], v[V];
    load_part(dy + c, d);
    load_part(x + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = r * (d[i] * load_w1(a.gamma, a.wtype, c + i, 1.f) - c1 - (v[i] - mu) * r * c2);
    store_part(dx + c, v);
  }
}

// (Runs before the kernel of dx, which may overwrite x or dy.)
template <typename X>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(const BwdArgs a) {
  let_next_start();
  wait_for_previous();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float dg = 0.f, db = 0.f;
#pragma unroll 8
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const float d = to_f(static_cast<const X*>(a.dy)[row * a.ld_dy + c]);
    const float x = to_f(static_cast<const X*>(a.x)[row * a.ld_x + c]);
    dg += d * ((x - a.mean[row]) * a.rstd[row]);
    db += d;
  }
  float* out = a.partial + (size_t)blockIdx.y * 2 * a.H;
  out[c] = dg;
  out[a.H + c] = db;
}

// ------------------------------------------------------------------ host
template <typename X>
cudaError_t backward_cols(const BwdArgs& a, int64_t max_blocks, int* blocks, cudaStream_t s) {
  if (!a.partial) return cudaSuccess;
  int64_t slabs = 64;
  if (slabs > a.T) slabs = a.T;
  if (slabs > max_blocks) slabs = max_blocks;
  *blocks = (int)slabs;
  return launch_overlapped(norm_bwd_cols_kernel<X>, dim3((a.H + 255) / 256, (unsigned)slabs), 256, 0, s, a);
}

template <typename X, int V>
cudaError_t backward_rows(const BwdArgs& a, int64_t max_blocks, int* blocks, cudaStream_t s) {
  const cudaError_t e = backward_cols<X>(a, max_blocks, blocks, s);
  if (e != cudaSuccess) return e;
  return launch_overlapped(norm_bwd_rows_kernel<X, V>, (unsigned)a.T, 1024, 0, s, a);
}

// Where the rows of a call's tensors start relative to 16-byte boundaries.
struct Offsets {
  bool vectors;   // all on boundaries, and rows are whole vectors
  bool same;      // at the same offset in every tensor, row by row
  int period;     // rows after which the offset repeats (1 .. 8)
};
Offsets offsets_of(const void* const* p, const int64_t* ld, int n, int es, int T, int H) {
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

template <typename X, bool SHIFT, int CPT, int L, int S>
cudaError_t run_fwd(const FwdArgs& a, const Offsets& o, cudaStream_t s) {
  static CtxCache<int> cache;
  constexpr int TH = kBlock<L, kFwdThreads>;
  constexpr int kBytes = Stream<X, CPT, L, SHIFT, S, TH>::RING + (CPT > 16 ? 2 * CPT * 4 * TH : 0);
  int blocks;
  return run(norm_fwd_kernel<X, SHIFT, CPT, L, S>, cache, a, kRows<L, kFwdThreads>, TH, kBytes, SHIFT ? o.period : 1,
             INT64_MAX, &blocks, s);
}

template <typename X, bool SHIFT, int CPT, int L, int S, bool GRADS = true>
cudaError_t run_bwd(const BwdArgs& a, const Offsets& o, int64_t max_blocks, int* blocks, cudaStream_t s) {
  static CtxCache<int> cache;
  constexpr int TH = kBlock<L, kBwdThreads<X>>;
  constexpr int kRing = 2 * Stream<X, CPT, L, SHIFT, S, TH>::RING + (CPT > 16 ? CPT * 4 * TH : 0);
  constexpr int kSums = kRows<L, kBwdThreads<X>> * 2 * L * CPT * 4;    // H <= L CPT
  return run(norm_bwd_kernel<X, SHIFT, CPT, L, S, GRADS>, cache, a, kRows<L, kBwdThreads<X>>, TH, kRing > kSums ? kRing : kSums,
             SHIFT ? o.period : 1, max_blocks, blocks, s);
}

// The first of these shapes that holds a row (with SHIFT, one from any place in
// its first vector): 16 lanes of 8 columns, a warp of 16 columns per lane, then
// whole warps of 16; 512 lanes of 32 columns for rows over 8192.  (Rows of 129 to
// 256 columns leave half of their warp idle: 65536 x 256 bf16 takes 16.7 us
// forward and 27.8 backward, 65536 x 512 24.0 and 39.6.)
// Over 8192 columns one block of 512 threads fits an SM, its ring holds two rows
// and the bf16 backward spills: 4000 x 9000 bf16 46 us forward and 91 backward
// (21 and 32 from HBM), 4000 x 9001 54 and 110; fp32 88 and 186 (42 and 64), its
// column sums from a read of their own.
template <typename X, bool SHIFT>
cudaError_t forward(const FwdArgs& a, const Offsets& o, cudaStream_t s) {
  const int n = SHIFT ? a.H + kVec<X> - 1 : a.H;
  if (n <= 128) return run_fwd<X, SHIFT, 8, 16, 4>(a, o, s);
  if (n <= 512) return run_fwd<X, SHIFT, 16, 32, 4>(a, o, s);
  if (n <= 1024) return run_fwd<X, SHIFT, 16, 64, 4>(a, o, s);
  if (n <= 1536) return run_fwd<X, SHIFT, 16, 96, 4>(a, o, s);
  if (n <= 2048) return run_fwd<X, SHIFT, 16, 128, 4>(a, o, s);
  if (n <= 2560) return run_fwd<X, SHIFT, 16, 160, 4>(a, o, s);
  if (n <= 3584) return run_fwd<X, SHIFT, 16, 224, 4>(a, o, s);
  if (n <= 4096) return run_fwd<X, SHIFT, 16, 256, 4>(a, o, s);
  if (n <= 5632) return run_fwd<X, SHIFT, 16, 352, 3>(a, o, s);
  if (n <= 8192) return run_fwd<X, SHIFT, 16, 512, 3>(a, o, s);
  if (n <= 16384) return run_fwd<X, SHIFT, 32, 512, sizeof(X) == 2 ? 2 : 1>(a, o, s);
  return launch_overlapped(norm_fwd_rows_kernel<X, SHIFT ? 1 : kVec<X>>, (unsigned)a.T, 1024, 0, s, a);
}

// As the forward.
template <typename X, bool SHIFT>
cudaError_t backward(const BwdArgs& a, const Offsets& o, int64_t max_blocks, int* blocks, cudaStream_t s) {
  constexpr bool B = sizeof(X) == 2;
  constexpr int S = B ? 4 : 3;
  const int n = SHIFT ? a.H + kVec<X> - 1 : a.H;
  if (n <= 128) return run_bwd<X, SHIFT, 8, 16, S>(a, o, max_blocks, blocks, s);
  if (n <= 512) return run_bwd<X, SHIFT, 16, 32, S>(a, o, max_blocks, blocks, s);
  if (n <= 1024) return run_bwd<X, SHIFT, 16, 64, S>(a, o, max_blocks, blocks, s);
  if (n <= 1536) return run_bwd<X, SHIFT, 16, 96, S>(a, o, max_blocks, blocks, s);
  if (n <= 2048) return run_bwd<X, SHIFT, 16, 128, S>(a, o, max_blocks, blocks, s);
  if (n <= 2560) return run_bwd<X, SHIFT, 16, 160, S>(a, o, max_blocks, blocks, s);
  if (n <= 3584) return run_bwd<X, SHIFT, 16, 224, S>(a, o, max_blocks, blocks, s);
  if (n <= 4096) return run_bwd<X, SHIFT, 16, 256, S>(a, o, max_blocks, blocks, s);
  if (n <= 5632) return run_bwd<X, SHIFT, 16, 352, 3>(a, o, max_blocks, blocks, s);
  if (n <= 8192) return run_bwd<X, SHIFT, 16, 512, 3>(a, o, max_blocks, blocks, s);
  if (n <= 16384) {
    if constexpr (B) {
      return run_bwd<X, SHIFT, 32, 512, 2>(a, o, max_blocks, blocks, s);
    } else {   // the ring holds one row of both tensors, and the registers no sums
      const cudaError_t e = backward_cols<X>(a, max_blocks, blocks, s);
      if (e != cudaSuccess) return e;
      int unused;
      return run_bwd<X, SHIFT, 32, 512, 1, false>(a, o, INT64_MAX, &unused, s);
    }
  }
  return backward_rows<X, SHIFT ? 1 : kVec<X>>(a, max_blocks, blocks, s);
}

template <typename X>
cudaError_t forward_any(const FwdArgs& a, const Offsets& o, cudaStream_t s) {
  if (o.vectors) return forward<X, false>(a, o, s);
  if (o.same) return forward<X, true>(a, o, s);
  return launch_overlapped(norm_fwd_rows_kernel<X, 1>, (unsigned)a.T, 1024, 0, s, a);
}

template <typename X>
cudaError_t backward_any(const BwdArgs& a, const Offsets& o, int64_t max_blocks, int* blocks, cudaStream_t s) {
  if (o.vectors) return backward<X, false>(a, o, max_blocks, blocks, s);
  if (o.same) return backward<X, true>(a, o, max_blocks, blocks, s);
  return backward_rows<X, 1>(a, max_blocks, blocks, s);
}

}  // namespace

cudaError_t launch_layer_norm(const NormDesc& d, const void* x, const void* gamma, const void* beta,
                              void* y, float* mean, float* rstd, cudaStream_t s) {
  const FwdArgs a{x, gamma, beta, y, mean, rstd, d.ld_x, d.ld_y, d.T, d.H, d.wtype, d.eps};
  const int es = d.xtype == MOE_TYPE_BF16 ? 2 : 4;
  const void* p[2] = {x, y};
  const int64_t ld[2] = {d.ld_x, d.ld_y};
  const Offsets o = offsets_of(p, ld, 2, es, d.T, d.H);
  return es == 2 ? forward_any<__nv_bfloat16>(a, o, s) : forward_any<float>(a, o, s);
}

int64_t norm_partial_blocks(int T) { return T < 1024 ? T : 1024; }

cudaError_t launch_layer_norm_backward(const NormDesc& d, const void* dy, const void* x,
                                       const void* gamma, const float* mean, const float* rstd,
                                       void* dx, void* dgamma, void* dbeta, float* partial,
                                       cudaStream_t s) {
  const bool params = dgamma || dbeta;
  const BwdArgs a{dy, x, gamma, mean, rstd, dx, params ? partial : nullptr, d.ld_y, d.ld_x, d.ld_dx,
                  d.T, d.H, d.wtype};
  const int es = d.xtype == MOE_TYPE_BF16 ? 2 : 4;
  int blocks = 0;
  if (d.T > 0) {
    const void* p[3] = {x, dy, dx};
    const int64_t ld[3] = {d.ld_x, d.ld_y, d.ld_dx};
    const Offsets o = offsets_of(p, ld, 3, es, d.T, d.H);
    const int64_t most = norm_partial_blocks(d.T);
    const cudaError_t e = es == 2 ? backward_any<__nv_bfloat16>(a, o, most, &blocks, s)
                                  : backward_any<float>(a, o, most, &blocks, s);
    if (e != cudaSuccess) return e;
  }
  if (params) {
    return launch_overlapped(norm_param_grad_kernel, dim3((d.H + 31) / 32, 2), 1024, 0, s,
                        (const float*)partial, blocks, d.H, d.wtype, dgamma, dbeta);
  }
  return cudaSuccess;
}

}  // namespace moe
