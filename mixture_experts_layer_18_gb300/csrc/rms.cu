// rms.cu - root-mean-square norm over the hidden axis with the residual's
// addition and an MXFP8 output, forward (rms_backward.cu: its backward).
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r gamma
//
// y in the type of x, as MXFP8 codes (blocks of 32 columns, the rule of
// quant.cu), or both; h in the type of x for the next residual addition and the
// backward.  Sum, statistics and y are fp32: y is taken from the sum before it is
// rounded to h, and its codes from y before it is rounded to y's type, so each
// result is rounded once.
//
// Bound by HBM: each of x, residual, h and y crosses it once, the codes at 33/64
// of a bf16 row.  Rows are held as rows.cuh describes; a block of 32 columns lies in 4
// (bf16) or 8 (fp32) neighbouring lanes, which join its maximum by shuffles.
//
// Measured (GB300): 16384 x 4096 bf16 with residual, h, y and codes 104 us (5.8 TB/s; two
// to six rows in the ring, two to four blocks per SM: 103 - 106); 5003 x 4096 fp32, the
// same, 53 us (6.6 TB/s); 5003 x 1999 fp32 in rows of 2001 28 us (5.7 TB/s); 4097 x 2048
// bf16, codes alone, 5.9 us; one row of 4096 1.9 us.
#include "mx_encode.cuh"
#include "rows.cuh"

namespace moe {

namespace {

using namespace rows;

constexpr int kThreads = 256;

struct RmsArgs {
  const void* x;
  const void* res;
  const void* gamma;
  void* h;
  void* y;
  uint8_t* q;
  uint8_t* sf;
  float* rstd;
  int64_t ld_x, ld_res, ld_h, ld_y;
  int T, H, wtype;
  float eps;
};

// Codes and scales of a lane's columns of one row (H a multiple of 32: a block
// is wholly in the row or past it).
template <typename X, int CPT, int L>
__device__ __forceinline__ void store_codes(const Lane<X, CPT, L, false>& l, uint8_t* q, uint8_t* sf, bool live,
                                            const F2 (&p)[CPT / 2]) {
  constexpr int V = kVec<X>;
#pragma unroll
  for (int j = 0; j < CPT / V; ++j) {
    float e[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) split(p[j * V / 2 + i], e[2 * i], e[2 * i + 1]);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, fabsf(e[i]));
#pragma unroll
    for (int o = 1; o < 32 / V; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int sb = mx_scale_byte(top);
    const float inv = mx_inv_scale(sb);
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      w[i] = e4m3x2(e[4 * i] * inv, e[4 * i + 1] * inv) |
             (uint32_t)e4m3x2(e[4 * i + 2] * inv, e[4 * i + 3] * inv) << 16;
    const int c = l.first() + j * L * V;
    if (live && l.valid(j)) {
      if constexpr (V == 8) *reinterpret_cast<uint2*>(q + c) = make_uint2(w[0], w[V / 4 - 1]);
      else *reinterpret_cast<uint32_t*>(q + c) = w[0];
      if (l.t % (32 / V) == 0) sf[c >> 5] = (uint8_t)sb;
    }
  }
}

template <typename X, bool SHIFT, bool RES, int CPT, int L, int S>
__global__ void __launch_bounds__(kBlock<L, kThreads>, CPT <= 16 ? 768 / kBlock<L, kThreads> : 1)
    rms_kernel(const __grid_constant__ RmsArgs a) {
  constexpr int TH = kBlock<L, kThreads>, ROWS = kRows<L, kThreads>;
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
  Str rs(lane, RES ? a.res : a.x, RES ? a.ld_res : a.ld_x, row, stride, dyn + (RES ? Str::RING : 0));
  wait_for_previous();
#pragma unroll
  for (int st = 0; st < S - 1; ++st) {
    xs.fetch(lane, row + st * stride, T, st);
    if (RES) rs.fetch(lane, row + st * stride, T, st);
    copy_commit();
  }
  Weights<X, CPT, L, SHIFT, TH> gam;
  gam.load(lane, a.gamma, a.wtype, 1.f, reinterpret_cast<float4*>(dyn + (RES ? 2 : 1) * Str::RING));
  int st = 0, par = 0;
  for (uint32_t base = blockIdx.x * ROWS; base < T; base += stride, row += stride) {
    F2 x[CPT / 2];
    const int to = st == 0 ? S - 1 : st - 1;
    xs.fetch(lane, row + (S - 1) * stride, T, to);
    if (RES) rs.fetch(lane, row + (S - 1) * stride, T, to);
    copy_commit();
    copy_wait<S - 1>();
    xs.take(lane, x, st);
    if (RES) {
      F2 d[CPT / 2];
      rs.take(lane, d, st);
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i) x[i] = add2(x[i], d[i]);
    }
    if (++st == S) st = 0;
    F2 acc = f2(0.f, 0.f), acc2 = acc;
#pragma unroll
    for (int i = 0; i < CPT / 2; i += 2) {
      acc = fma2(x[i], x[i], acc);
      acc2 = fma2(x[i + 1], x[i + 1], acc2);
    }
    float s[1] = {sum2(add2(acc, acc2))};
    row_sums<1, L>(s, group, sm[par]);
    par ^= 1;
    const float r = inv_sqrt_exact(s[0] / (float)a.H + a.eps);
    const bool live = row < T;
    if (RES && a.h && live) store_row(lane, static_cast<X*>(a.h) + (int64_t)row * a.ld_h, x);
    F2 g[CPT / 2];
    gam.get(g);
    const F2 rr = f2(r, r);
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) x[i] = mul2(mul2(x[i], rr), g[i]);
    if (a.y && live) store_row(lane, static_cast<X*>(a.y) + (int64_t)row * a.ld_y, x);
    if constexpr (!SHIFT)
      if (a.q) store_codes(lane, a.q + (int64_t)row * a.H, a.sf + (int64_t)row * (a.H >> 5), live, x);
    if (live && lane.t == 0 && a.rstd) a.rstd[row] = r;
  }
  copy_wait<0>();
}

// Rows that the kernel above does not take (longer than 16384, tensors at
// different offsets from 16-byte boundaries, codes of rows off them): a block
// per row, two passes over it; by vectors where all rows start on 16-byte
// boundaries, by blocks of 32 columns where there are codes, else by elements.
template <typename X, int V>
__global__ void __launch_bounds__(1024) rms_rows_kernel(const RmsArgs a) {
  __shared__ float sm[32];
  let_next_start();
  wait_for_previous();
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  const X* res = a.res ? static_cast<const X*>(a.res) + row * a.ld_res : nullptr;
  X* h = a.h ? static_cast<X*>(a.h) + row * a.ld_h : nullptr;
  X* y = a.y ? static_cast<X*>(a.y) + row * a.ld_y : nullptr;
  auto sum_of = [&](int c, float (&v)[V]) {
    load_part(x + c, v);
    if (res) {
      float d[V];
      load_part(res + c, d);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += d[i];
    }
  };
  float s[1] = {0.f};
#pragma unroll 4
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float v[V];
    sum_of(c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] += v[i] * v[i];
  }
  row_sums<1, 1024>(s, 0, sm);
  const float r = inv_sqrt_exact(s[0] / (float)a.H + a.eps);
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
  auto part = [&](int c, float (&v)[V]) {        // stores h and y of V columns; v: y
    sum_of(c, v);
    if (res && h) store_part(h + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = v[i] * r * load_w1(a.gamma, a.wtype, c + i, 1.f);
    if (y) store_part(y + c, v);
  };
  if (!a.q) {
#pragma unroll 2
    for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
      float v[V];
      part(c, v);
    }
    return;
  }
  for (int b = threadIdx.x; b < a.H / 32; b += 1024) {
    float e[32], top = 0.f;
#pragma unroll
    for (int i = 0; i < 32 / V; ++i) {
      float v[V];
      part(b * 32 + i * V, v);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        e[i * V + k] = v[k];
        top = fmaxf(top, fabsf(v[k]));
      }
    }
    const int sb = mx_scale_byte(top);
    const float inv = mx_inv_scale(sb);
    uint4* q = reinterpret_cast<uint4*>(a.q + row * a.H + b * 32);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float* f = e + i * 16 + k * 4;
        w[k] = e4m3x2(f[0] * inv, f[1] * inv) | (uint32_t)e4m3x2(f[2] * inv, f[3] * inv) << 16;
      }
      q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    a.sf[row * (a.H / 32) + b] = (uint8_t)sb;
  }
}

template <typename X, bool SHIFT, bool RES, int CPT, int L, int S>
cudaError_t run_rms(const RmsArgs& a, const Offsets& o, cudaStream_t s) {
  static CtxCache<int> cache;
  constexpr int TH = kBlock<L, kThreads>;
  constexpr int kBytes = (RES ? 2 : 1) * Stream<X, CPT, L, SHIFT, S, TH>::RING + (CPT > 16 ? CPT * 4 * TH : 0);
  int blocks;
  return run(rms_kernel<X, SHIFT, RES, CPT, L, S>, cache, a, kRows<L, kThreads>, TH, kBytes, SHIFT ? o.period : 1,
             INT64_MAX, &blocks, s);
}

// The shapes of the layer norm's rows; the ring holds as many rows as the two
// tensors leave room for.
template <typename X, bool SHIFT, bool RES>
cudaError_t rms_shape(const RmsArgs& a, const Offsets& o, cudaStream_t s) {
  constexpr bool B = sizeof(X) == 2;
  const int n = SHIFT ? a.H + kVec<X> - 1 : a.H;
  if (n <= 128) return run_rms<X, SHIFT, RES, 8, 16, 4>(a, o, s);
  if (n <= 512) return run_rms<X, SHIFT, RES, 16, 32, 4>(a, o, s);
  if (n <= 1024) return run_rms<X, SHIFT, RES, 16, 64, 4>(a, o, s);
  if (n <= 1536) return run_rms<X, SHIFT, RES, 16, 96, 4>(a, o, s);
  if (n <= 2048) return run_rms<X, SHIFT, RES, 16, 128, 4>(a, o, s);
  if (n <= 2560) return run_rms<X, SHIFT, RES, 16, 160, 4>(a, o, s);
  if (n <= 3584) return run_rms<X, SHIFT, RES, 16, 224, 4>(a, o, s);
  if (n <= 4096) return run_rms<X, SHIFT, RES, 16, 256, 4>(a, o, s);
  if (n <= 5632) return run_rms<X, SHIFT, RES, 16, 352, 3>(a, o, s);
  if (n <= 8192) return run_rms<X, SHIFT, RES, 16, 512, 3>(a, o, s);
  if (n <= 16384) return run_rms<X, SHIFT, RES, 32, 512, B ? 2 : 1>(a, o, s);
  return launch_overlapped(rms_rows_kernel<X, SHIFT ? 1 : kVec<X>>, (unsigned)a.T, 1024, 0, s, a);
}

template <typename X>
cudaError_t rms_any(const RmsArgs& a, const Offsets& o, cudaStream_t s) {
  if (o.vectors) return a.res ? rms_shape<X, false, true>(a, o, s) : rms_shape<X, false, false>(a, o, s);
  if (o.same && !a.q) return a.res ? rms_shape<X, true, true>(a, o, s) : rms_shape<X, true, false>(a, o, s);
  return launch_overlapped(rms_rows_kernel<X, 1>, (unsigned)a.T, 1024, 0, s, a);
}

}  // namespace

cudaError_t launch_rms_norm(const moe_rms_dims& d, const void* x, const void* res, const void* gamma, void* h,
                            void* y, uint8_t* q, uint8_t* sf, float* rstd, cudaStream_t s) {
  if (!res) h = nullptr;
  const RmsArgs a{x, res, gamma, h, y, q, sf, rstd, d.ld_x, d.ld_residual, d.ld_h, d.ld_y, d.T, d.H, d.w_type, d.eps};
  const void* p[4] = {x};
  int64_t ld[4] = {d.ld_x};
  int n = 1;
  if (res) p[n] = res, ld[n++] = d.ld_residual;
  if (h) p[n] = h, ld[n++] = d.ld_h;
  if (y) p[n] = y, ld[n++] = d.ld_y;
  const int es = d.x_type == MOE_TYPE_BF16 ? 2 : 4;
  const Offsets o = offsets_of(p, ld, n, es, d.T, d.H);
  return es == 2 ? rms_any<__nv_bfloat16>(a, o, s) : rms_any<float>(a, o, s);
}

}  // namespace moe
