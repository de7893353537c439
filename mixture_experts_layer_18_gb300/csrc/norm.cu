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
// Blocks are persistent.  Where every row starts on a 16-byte boundary, a
// lane's vectors of the next rows travel to its own slots of shared memory
// (asynchronous copies that only this lane reads, so no barrier orders them);
// otherwise (odd widths or strides) lanes load single elements, the next
// row's into registers.  L and the columns per lane are compile-time numbers:
// a row's offsets are then part of the instructions, which with the arithmetic
// in pairs (fp32x2) keeps a row's instructions below the time that HBM takes
// for it (they were the bound of a first version with both at run time).
// Columns past the row's end read as zero; a group past the last row works on
// what its slots hold and stores nothing.
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
    const int k = lane / W, w = lane & (W - 1);
    const float* g = sm + group * WARPS * N;
    x = w < WARPS ? g[w * N + k] : 0.f;
    if constexpr (WARPS > W) x += g[(w + W) * N + k];
    x = lanes_sum<W>(x);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = N == 1 ? x : __shfl_sync(0xffffffffu, x, i * W);
  }
}

// 1 / sqrt(v): the approximation and one Newton step (below one ulp of fp32).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  // v = 0 gives infinity, which the step would turn into NaN
  return v > 0.f ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
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

// A lane's CPT columns of every row, V to a load: element i of load j is
// column (j L + t) V + i.  V is the row's vector (16 bytes) or one element.
template <typename X, int V, int CPT, int L>
struct Lane {
  int t, left;                           // `left`: columns from this lane's first to the row's end
  __device__ __forceinline__ Lane(int H) : t(threadIdx.x & (L - 1)), left(H - t * V) {}
  __device__ __forceinline__ bool valid(int j) const { return left > j * L * V; }
  __device__ __forceinline__ int first() const { return t * V; }
};

// Load j of a lane, as pairs, to its place in a row; a whole part of a row.
template <typename X, int V, int CPT, int L>
__device__ __forceinline__ void store_vec(const Lane<X, V, CPT, L>& l, X* row, int j, const F2* p) {
  static_assert(V > 1, "vectors");
  float e[V];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) split(p[i], e[2 * i], e[2 * i + 1]);
  X* q = row + l.first() + j * L * V;
  if (!l.valid(j)) return;
  if constexpr (sizeof(X) == 2)
    *reinterpret_cast<uint4*>(q) = make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]),
                                              pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7]));
  else
    *reinterpret_cast<float4*>(q) = make_float4(e[0], e[1], e[2], e[3]);
}
template <typename X, int V, int CPT, int L>
__device__ __forceinline__ void store_row(const Lane<X, V, CPT, L>& l, X* row, const F2 (&p)[CPT / 2]) {
  if constexpr (V > 1) {
#pragma unroll
    for (int j = 0; j < CPT / V; ++j) store_vec(l, row, j, p + j * V / 2);
  } else {
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      float e[2];
      split(p[j / 2], e[0], e[1]);
      if (l.valid(j)) put(row + l.first() + j * L, e[j & 1]);
    }
  }
}

// A lane's weights, read once per block (0 past the row's end): in registers
// up to 16 columns, else in shared memory (each lane's own, 16 bytes apart).
template <typename X, int V, int CPT, int L, int THREADS>
struct Weights {
  static constexpr bool REGS = CPT <= 16;
  F2 r[REGS ? CPT / 2 : 1];
  float4* s;
  __device__ __forceinline__ void load(const Lane<X, V, CPT, L>& l, const void* p, int type, float fill,
                                       float4* smem) {
    s = smem + threadIdx.x;
    F2 v[CPT / 2];
#pragma unroll
    for (int j = 0; j < CPT / V; ++j) {
      float e[V] = {};
      const int c = l.first() + j * L * V;
      if (l.valid(j)) {
        if (V == 8 && p && type == MOE_TYPE_BF16 && ((uintptr_t)p & 15) == 0) {
          const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + c);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < V; ++i) e[i] = i & 1 ? bf16_hi(w[(i / 2) & 3]) : bf16_lo(w[(i / 2) & 3]);
        } else if (V >= 4 && p && type == MOE_TYPE_F32 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
          for (int i = 0; i + 3 < V; i += 4) {
            const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + i);
            e[i] = u.x; e[i + 1] = u.y; e[i + 2] = u.z; e[i + 3] = u.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) e[i] = load_w1(p, type, c + i, fill);
        }
      }
      if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[j * V / 2 + i] = f2(e[2 * i], e[2 * i + 1]);
      } else if (j & 1) {
        float a, b;
        split(v[j / 2], a, b);
        v[j / 2] = f2(a, e[0]);
      } else {
        v[j / 2] = f2(e[0], 0.f);
      }
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

// The rows of one tensor on their way to a lane.  Vectors: a ring of S rows
// in shared memory, `at` the lane's first slot.  Elements: the next row in
// registers.  Slots (registers) past the row's end are zero from the start
// and never written.
template <typename X, int V, int CPT, int L, int S, int THREADS>
struct Stream {
  static constexpr int NL = CPT / V;
  static constexpr int RING = V == 1 ? 0 : S * NL * THREADS * 16;    // bytes per block
  const X* p;
  int64_t ld;
  uint8_t* at;
  X next[V == 1 ? CPT : 1];
  __device__ __forceinline__ Stream(const Lane<X, V, CPT, L>& l, const void* base, int64_t ld_, uint8_t* ring)
      : p(static_cast<const X*>(base) + l.first()), ld(ld_), at(ring + threadIdx.x * 16) {
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) put(&next[i], 0.f);
    } else {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if (!l.valid(j))
          for (int st = 0; st < S; ++st)
            *reinterpret_cast<uint4*>(at + (st * NL + j) * THREADS * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void fetch(const Lane<X, V, CPT, L>& l, int64_t row, int T, int st) {
    if (row >= T) return;
    const X* q = p + row * ld;
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 0; i < CPT; ++i)
        if (l.valid(i)) next[i] = q[i * L];
    } else {
      const uint32_t d = smem_u32(at) + st * (NL * THREADS * 16);
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if (l.valid(j)) copy_async16(d + j * THREADS * 16, q + j * L * V);
    }
  }
  __device__ __forceinline__ void take(F2 (&x)[CPT / 2], int st) const {
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i) x[i] = f2(to_f(next[2 * i]), to_f(next[2 * i + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const uint4 u = *reinterpret_cast<const uint4*>(at + (st * NL + j) * THREADS * 16);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
          x[j * V / 2 + i] = sizeof(X) == 2
                                 ? f2(bf16_lo(w[i]), bf16_hi(w[i]))
                                 : f2(__uint_as_float(w[(2 * i) & 3]), __uint_as_float(w[(2 * i + 1) & 3]));
      }
    }
  }
};

template <int L>
constexpr int kRows = L >= 256 ? 1 : 256 / L;     // rows of a block
template <int L>
constexpr int kBlock = kRows<L>* L;

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

template <typename X, int V, int CPT, int L, int S>
__global__ void __launch_bounds__(kBlock<L>, kBlock<L> == 256 && CPT <= 16 ? 3 : 1)
    norm_fwd_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int TH = kBlock<L>, ROWS = kRows<L>;
  using Str = Stream<X, V, CPT, L, S, TH>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float sm[2][TH / 32];
  const int group = threadIdx.x / L;
  const Lane<X, V, CPT, L> lane(a.H);
  const int64_t stride = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + group;
  Str xs(lane, a.x, a.ld_x, dyn);
#pragma unroll
  for (int st = 0; st < (V == 1 ? 1 : S - 1); ++st) {
    xs.fetch(lane, row + st * stride, a.T, st);
    copy_commit();
  }
  Weights<X, V, CPT, L, TH> gam, bet;
  float4* wsm = reinterpret_cast<float4*>(dyn + Str::RING);
  gam.load(lane, a.gamma, a.wtype, 1.f, wsm);
  bet.load(lane, a.beta, a.wtype, 0.f, wsm + CPT / 4 * TH);
  const float inv = 1.f / (float)a.H;
  int st = 0;
  for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.T; base += stride, row += stride) {
    F2 x[CPT / 2];
    if constexpr (V > 1) {
      xs.fetch(lane, row + (S - 1) * stride, a.T, st == 0 ? S - 1 : st - 1);
      copy_commit();
      copy_wait<S - 1>();
    }
    xs.take(x, st);
    if constexpr (V == 1) xs.fetch(lane, row + stride, a.T, 0);
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
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i) {
        float d, e;
        split(x[i], d, e);
        q[0] += lane.valid(2 * i) ? d * d : 0.f;
        q[0] += lane.valid(2 * i + 1) ? e * e : 0.f;
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
    if (row < a.T) {
      store_row(lane, static_cast<X*>(a.y) + row * a.ld_y, x);
      if (lane.t == 0) {
        if (a.mean) a.mean[row] = mu;
        if (a.rstd) a.rstd[row] = r;
      }
    }
  }
  copy_wait<0>();
}

// Rows too long for the kernel above: a block per row, three passes over it
// (the second and third find most of it in L1 or L2).
template <typename X>
__global__ void __launch_bounds__(1024) norm_fwd_rows_kernel(const FwdArgs a) {
  __shared__ float sm[2][32];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  float s[1] = {0.f}, q[1] = {0.f};
  for (int c = threadIdx.x; c < a.H; c += blockDim.x) s[0] += to_f(x[c]);
  row_sums<1, 1024>(s, 0, sm[0]);
  const float mu = s[0] / (float)a.H;
  for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
    const float d = to_f(x[c]) - mu;
    q[0] += d * d;
  }
  row_sums<1, 1024>(q, 0, sm[1]);
  const float r = 1.f / sqrtf(q[0] / (float)a.H + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  X* y = static_cast<X*>(a.y) + row * a.ld_y;
  for (int c = threadIdx.x; c < a.H; c += blockDim.x)
    put(y + c, (to_f(x[c]) - mu) * r * load_w1(a.gamma, a.wtype, c, 1.f) + load_w1(a.beta, a.wtype, c, 0.f));
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
template <typename X, int V, int CPT, int L, int S>
__global__ void __launch_bounds__(kBlock<L>, kBlock<L> == 256 && CPT <= 16 ? 2 : 1)
    norm_bwd_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int TH = kBlock<L>, ROWS = kRows<L>;
  using Str = Stream<X, V, CPT, L, S, TH>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float sm[2][TH / 16];
  let_next_start();
  const int group = threadIdx.x / L;
  const Lane<X, V, CPT, L> lane(a.H);
  const int64_t stride = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + group;
  Str xs(lane, a.x, a.ld_x, dyn), ds(lane, a.dy, a.ld_dy, dyn + Str::RING);
#pragma unroll
  for (int st = 0; st < (V == 1 ? 1 : S - 1); ++st) {
    xs.fetch(lane, row + st * stride, a.T, st);
    ds.fetch(lane, row + st * stride, a.T, st);
    copy_commit();
  }
  auto at = [&](int64_t q) { return q < a.T ? q : a.T - 1; };
  float mu = a.mean[at(row)], r = a.rstd[at(row)];
  Weights<X, V, CPT, L, TH> gam;
  gam.load(lane, a.gamma, a.wtype, 1.f, reinterpret_cast<float4*>(dyn + 2 * Str::RING));
  F2 dg[CPT / 2], db[CPT / 2];
#pragma unroll
  for (int i = 0; i < CPT / 2; ++i) dg[i] = db[i] = f2(0.f, 0.f);
  const float inv = 1.f / (float)a.H;
  int st = 0, par = 0;
  for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.T; base += stride, row += stride) {
    const float rc = r, bc = -mu * r;
    const bool live = row < a.T;
    mu = a.mean[at(row + stride)];
    r = a.rstd[at(row + stride)];
    if constexpr (V > 1) {
      const int to = st == 0 ? S - 1 : st - 1;
      xs.fetch(lane, row + (S - 1) * stride, a.T, to);
      ds.fetch(lane, row + (S - 1) * stride, a.T, to);
      copy_commit();
      copy_wait<S - 1>();
    }
    const F2 rr = f2(rc, rc), bb = f2(bc, bc);
    F2 s1 = f2(0.f, 0.f), s2 = s1;
    F2 x[CPT / 2], d[CPT / 2], g[CPT / 2];
    xs.take(x, st);
    ds.take(d, st);
    if (++st == S) st = 0;
    gam.get(g);
    if constexpr (V == 1) {
      xs.fetch(lane, row + stride, a.T, 0);
      ds.fetch(lane, row + stride, a.T, 0);
    }
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) {
      const F2 h = fma2(x[i], rr, bb);
      const F2 gy = mul2(d[i], g[i]);
      s1 = add2(s1, gy);
      s2 = fma2(gy, h, s2);
      if (live) {
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
    if (live) store_row(lane, static_cast<X*>(a.dx) + row * a.ld_dx, x);
  }
  copy_wait<0>();
  if (!a.partial) return;
  // the block's column sums: groups of one block are added in order
  float* out = a.partial + (size_t)blockIdx.x * 2 * a.H;
  float* acc = reinterpret_cast<float*>(dyn) + (size_t)group * 2 * a.H;   // [ROWS][2][H]
  if (ROWS > 1) __syncthreads();         // the ring is no longer read
#pragma unroll
  for (int i = 0; i < CPT / 2; ++i) {
    float gs[2], bs[2];
    split(dg[i], gs[0], gs[1]);
    split(db[i], bs[0], bs[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = (2 * i + k) / V, c = lane.first() + j * L * V + (2 * i + k) % V;
      if (!lane.valid(j)) continue;
      if constexpr (ROWS == 1) {
        out[c] = gs[k];
        out[a.H + c] = bs[k];
      } else {
        acc[c] = gs[k];
        acc[a.H + c] = bs[k];
      }
    }
  }
  if constexpr (ROWS > 1) {
    __syncthreads();
    const float* all = reinterpret_cast<const float*>(dyn);
    for (int c = threadIdx.x; c < 2 * a.H; c += TH) {
      float v = 0.f;
      for (int g = 0; g < ROWS; ++g) v += all[(size_t)2 * g * a.H + c];
      out[c] = v;
    }
  }
}

// dgamma and dbeta from the blocks' partial sums: 32 columns per block, 32
// slices of the partials, added as a fixed tree.
__global__ void __launch_bounds__(1024) norm_param_grad_kernel(const float* partial, int blocks, int H,
                                                               int wtype, void* dgamma, void* dbeta) {
  __shared__ float sm[32][33];
  wait_for_previous();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H)
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

// Rows too long for the kernel above: dx with a block per row (two passes),
// the column sums from a second read with a thread per column.
template <typename X>
__global__ void __launch_bounds__(1024) norm_bwd_rows_kernel(const BwdArgs a) {
  __shared__ float sm[64];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  const X* dy = static_cast<const X*>(a.dy) + row * a.ld_dy;
  const float mu = a.mean[row], r = a.rstd[row];
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
    const float gy = to_f(dy[c]) * load_w1(a.gamma, a.wtype, c, 1.f);
    s[0] += gy;
    s[1] += gy * ((to_f(x[c]) - mu) * r);
  }
  row_sums<2, 1024>(s, 0, sm);
  const float c1 = s[0] / (float)a.H, c2 = s[1] / (float)a.H;
  X* dx = static_cast<X*>(a.dx) + row * a.ld_dx;
  for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
    const float gy = to_f(dy[c]) * load_w1(a.gamma, a.wtype, c, 1.f);
    put(dx + c, r * (gy - c1 - (to_f(x[c]) - mu) * r * c2));
  }
}

// Before the rows kernel: dx may overwrite x or dy.
template <typename X>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(const BwdArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float dg = 0.f, db = 0.f;
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
// Launches one form: blocks that fill the GPU once, but no more than there
// are rows.
template <typename Args, typename K>
cudaError_t run(K kern, CtxCache<int>& cache, const Args& a, int rows, int threads, int smem,
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
  if (blocks > need) blocks = need;
  if (blocks > max_blocks) blocks = max_blocks;
  kern<<<(unsigned)blocks, threads, smem, s>>>(a);
  *blocks_out = (int)blocks;
  return cudaGetLastError();
}

template <typename X, int V, int CPT, int L, int S>
cudaError_t run_fwd(const FwdArgs& a, cudaStream_t s) {
  static CtxCache<int> cache;
  constexpr int TH = kBlock<L>;
  constexpr int kBytes = Stream<X, V, CPT, L, S, TH>::RING + (CPT > 16 ? 2 * CPT * 4 * TH : 0);
  int blocks;
  return run(norm_fwd_kernel<X, V, CPT, L, S>, cache, a, kRows<L>, TH, kBytes, INT64_MAX, &blocks, s);
}

template <typename X, int V, int CPT, int L, int S>
cudaError_t run_bwd(const BwdArgs& a, int64_t max_blocks, int* blocks, cudaStream_t s) {
  static CtxCache<int> cache;
  constexpr int TH = kBlock<L>;
  constexpr int kRing = 2 * Stream<X, V, CPT, L, S, TH>::RING + (CPT > 16 ? CPT * 4 * TH : 0);
  constexpr int kSums = kRows<L> > 1 ? kRows<L> * 2 * L * CPT * 4 : 0;    // H <= L CPT
  return run(norm_bwd_kernel<X, V, CPT, L, S>, cache, a, kRows<L>, TH, kRing > kSums ? kRing : kSums,
             max_blocks, blocks, s);
}

// The fewest lanes that hold a row at 16 columns each (8 in rows up to 128 and
// where lanes load single elements, whose next row sits in registers), 512
// lanes of 32 columns (vectors only) for rows over 8192.
template <typename X, int V>
cudaError_t forward(const FwdArgs& a, cudaStream_t s) {
  constexpr bool B = sizeof(X) == 2;
  constexpr int C = V == 1 ? 8 : 16;
  if (a.H <= 128) return run_fwd<X, V, 8, 16, 4>(a, s);
  if (a.H <= 32 * C) return run_fwd<X, V, C, 32, 4>(a, s);
  if (a.H <= 64 * C) return run_fwd<X, V, C, 64, 4>(a, s);
  if (a.H <= 128 * C) return run_fwd<X, V, C, 128, 4>(a, s);
  if (a.H <= 256 * C) return run_fwd<X, V, C, 256, 4>(a, s);
  if (a.H <= 4096) return run_fwd<X, V, 16, 256, 4>(a, s);
  if (a.H <= 8192) return run_fwd<X, V, 16, 512, 3>(a, s);
  if constexpr (V > 1)
    if (a.H <= 16384) return run_fwd<X, V, 32, 512, B ? 2 : 1>(a, s);
  norm_fwd_rows_kernel<X><<<(unsigned)a.T, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

// As the forward; fp32 rows over 8192 would not fit the ring with two tensors.
template <typename X, int V>
cudaError_t backward(const BwdArgs& a, int64_t max_blocks, int* blocks, cudaStream_t s) {
  constexpr bool B = sizeof(X) == 2;
  constexpr int S = B ? 4 : 3;
  constexpr int C = V == 1 ? 8 : 16;
  if (a.H <= 128) return run_bwd<X, V, 8, 16, S>(a, max_blocks, blocks, s);
  if (a.H <= 32 * C) return run_bwd<X, V, C, 32, S>(a, max_blocks, blocks, s);
  if (a.H <= 64 * C) return run_bwd<X, V, C, 64, S>(a, max_blocks, blocks, s);
  if (a.H <= 128 * C) return run_bwd<X, V, C, 128, S>(a, max_blocks, blocks, s);
  if (a.H <= 256 * C) return run_bwd<X, V, C, 256, S>(a, max_blocks, blocks, s);
  if (a.H <= 512 * C && C == 8) return run_bwd<X, V, C, 512, S>(a, max_blocks, blocks, s);
  if (a.H <= 8192) return run_bwd<X, V, 16, 512, 3>(a, max_blocks, blocks, s);
  if constexpr (B && (V > 1))
    if (a.H <= 16384) return run_bwd<X, V, 32, 512, 2>(a, max_blocks, blocks, s);
  if (a.partial) {
    int64_t slabs = 64;
    if (slabs > a.T) slabs = a.T;
    if (slabs > max_blocks) slabs = max_blocks;
    norm_bwd_cols_kernel<X><<<dim3((a.H + 255) / 256, (unsigned)slabs), 256, 0, s>>>(a);
    *blocks = (int)slabs;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_bwd_rows_kernel<X><<<(unsigned)a.T, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

bool rows16(const void* p, int64_t ld, int T, int es) {
  return ((uintptr_t)p & 15) == 0 && (T <= 1 || (ld * es) % 16 == 0);
}

}  // namespace

cudaError_t launch_layer_norm(const NormDesc& d, const void* x, const void* gamma, const void* beta,
                              void* y, float* mean, float* rstd, cudaStream_t s) {
  FwdArgs a{x, gamma, beta, y, mean, rstd, d.ld_x, d.ld_y, d.T, d.H, d.wtype, d.eps};
  const int es = d.xtype == MOE_TYPE_BF16 ? 2 : 4;
  const bool vec = ((int64_t)d.H * es) % 16 == 0 && rows16(x, d.ld_x, d.T, es) && rows16(y, d.ld_y, d.T, es);
  if (es == 2) return vec ? forward<__nv_bfloat16, 8>(a, s) : forward<__nv_bfloat16, 1>(a, s);
  return vec ? forward<float, 4>(a, s) : forward<float, 1>(a, s);
}

int64_t norm_partial_blocks(int T) { return T < 1024 ? T : 1024; }

cudaError_t launch_layer_norm_backward(const NormDesc& d, const void* dy, const void* x,
                                       const void* gamma, const float* mean, const float* rstd,
                                       void* dx, void* dgamma, void* dbeta, float* partial,
                                       cudaStream_t s) {
  const bool params = dgamma || dbeta;
  BwdArgs a{dy, x, gamma, mean, rstd, dx, params ? partial : nullptr, d.ld_y, d.ld_x, d.ld_dx,
            d.T, d.H, d.wtype};
  const int es = d.xtype == MOE_TYPE_BF16 ? 2 : 4;
  int blocks = 0;
  if (d.T > 0) {
    const bool vec = ((int64_t)d.H * es) % 16 == 0 && rows16(x, d.ld_x, d.T, es) &&
                     rows16(dy, d.ld_y, d.T, es) && rows16(dx, d.ld_dx, d.T, es);
    const int64_t most = norm_partial_blocks(d.T);
    cudaError_t e;
    if (es == 2)
      e = vec ? backward<__nv_bfloat16, 8>(a, most, &blocks, s) : backward<__nv_bfloat16, 1>(a, most, &blocks, s);
    else
      e = vec ? backward<float, 4>(a, most, &blocks, s) : backward<float, 1>(a, most, &blocks, s);
    if (e != cudaSuccess) return e;
  }
  if (params) {
    return launch_after(norm_param_grad_kernel, dim3((d.H + 31) / 32, 2), 1024, 0, s,
                        (const float*)partial, blocks, d.H, d.wtype, dgamma, dbeta);
  }
  return cudaSuccess;
}

}  // namespace moe
