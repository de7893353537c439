// rms_backward.cu - backward of the root-mean-square norm with the residual's
// addition (rms.cu).
//
//   xh = h r, g = gamma dy:
//   dx = r g - h r^2 mean(g xh) + dh,   dgamma = sum over rows of dy xh
//
// dh is the gradient that reaches the sum h directly (the residual path); dx is
// the gradient of x and of the residual alike.  Bound by HBM: dy, h and dh are read
// once, dx is written once.  Rows are held as rows.cuh describes; the column sums of
// dgamma stay in registers over all rows of a block, are joined in shared memory and
// added up over the blocks by a second kernel, in a fixed order.
//
// Measured (GB300), with dh and dgamma: 16384 x 4096 bf16 79 us (6.8 TB/s: part of it
// from L2); 5003 x 4096 fp32 52 us (6.3 TB/s), 5003 x 1999 in rows of 2001 32 us (5.0
// TB/s; two rows in the ring instead of three 33.6); the second kernel is 2 - 5 us of these.
#include "rows.cuh"

namespace moe {

namespace {

using namespace rows;

template <typename X>
constexpr int kThreads = sizeof(X) == 2 ? 512 : 256;

struct RmsBwdArgs {
  const void* dy;
  const void* h;
  const void* dh;
  const void* gamma;
  const float* rstd;
  void* dx;
  float* partial;      // [blocks][H]: dgamma sums of each block
  int64_t ld_dy, ld_h, ld_dh, ld_dx;
  int T, H, wtype;
};

// A lane's columns of a row straight from memory (0 past its ends).
template <typename X, int CPT, int L, bool SHIFT>
__device__ __forceinline__ void add_row(const Lane<X, CPT, L, SHIFT>& l, const X* row, F2 (&x)[CPT / 2]) {
  constexpr int V = kVec<X>;
  row += l.first();
#pragma unroll
  for (int j = 0; j < CPT / V; ++j) {
    float e[V] = {};
    if (l.full(j)) {
      load_part(row + j * L * V, e);
    } else if (SHIFT && l.valid(j)) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (l.inside(j, i)) e[i] = to_f(row[j * L * V + i]);
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) x[j * V / 2 + i] = add2(x[j * V / 2 + i], f2(e[2 * i], e[2 * i + 1]));
  }
}

// GRADS: with the column sums of dgamma.  DH: dh travels through a ring of its own
// (rows of 32 columns per lane leave no room for one and read it from memory).
template <typename X, bool SHIFT, bool DH, int CPT, int L, int S, bool GRADS>
__global__ void __launch_bounds__(kBlock<L, kThreads<X>>, CPT <= 16 ? 512 / kBlock<L, kThreads<X>> : 1)
    rms_bwd_kernel(const __grid_constant__ RmsBwdArgs a) {
  constexpr int TH = kBlock<L, kThreads<X>>, ROWS = kRows<L, kThreads<X>>, V = kVec<X>;
  constexpr bool RING = DH && CPT <= 16;
  using Str = Stream<X, CPT, L, SHIFT, S, TH>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float sm[2][TH / 32];
  let_next_start();
  const int group = threadIdx.x / L;
  const uint32_t T = a.T, stride = gridDim.x * ROWS;   // (T below 2^31: rows past it do not wrap)
  uint32_t row = blockIdx.x * ROWS + group;
  const Lane<X, CPT, L, SHIFT> lane(
      a.H, SHIFT ? shift_of(static_cast<const X*>(a.h) + (row < T ? row : 0) * a.ld_h) : 0);
  Str hs(lane, a.h, a.ld_h, row, stride, dyn), ds(lane, a.dy, a.ld_dy, row, stride, dyn + Str::RING);
  Str es(lane, RING ? a.dh : a.h, RING ? a.ld_dh : a.ld_h, row, stride, dyn + (RING ? 2 * Str::RING : 0));
  X* dx = static_cast<X*>(a.dx) + row * a.ld_dx;
  const int64_t dx_step = stride * a.ld_dx;
  wait_for_previous();
#pragma unroll
  for (int st = 0; st < S - 1; ++st) {
    hs.fetch(lane, row + st * stride, T, st);
    ds.fetch(lane, row + st * stride, T, st);
    if (RING) es.fetch(lane, row + st * stride, T, st);
    copy_commit();
  }
  auto at = [&](uint32_t q) { return q < T ? q : T - 1; };
  float r = a.rstd[at(row)];
  Weights<X, CPT, L, SHIFT, TH> gam;
  gam.load(lane, a.gamma, a.wtype, 1.f, reinterpret_cast<float4*>(dyn + (RING ? 3 : 2) * Str::RING));
  F2 dg[CPT / 2];
#pragma unroll
  for (int i = 0; i < CPT / 2; ++i) dg[i] = f2(0.f, 0.f);
  const float inv = 1.f / (float)a.H;
  int st = 0, par = 0;
  for (uint32_t base = blockIdx.x * ROWS; base < T; base += stride, row += stride) {
    const float rc = r;
    const bool live = row < T;
    r = a.rstd[at(row + stride)];
    const int to = st == 0 ? S - 1 : st - 1;
    hs.fetch(lane, row + (S - 1) * stride, T, to);
    ds.fetch(lane, row + (S - 1) * stride, T, to);
    if (RING) es.fetch(lane, row + (S - 1) * stride, T, to);
    copy_commit();
    copy_wait<S - 1>();
    const F2 rr = f2(rc, rc);
    F2 s2 = f2(0.f, 0.f);
    F2 x[CPT / 2], d[CPT / 2], g[CPT / 2];
    hs.take(lane, x, st);
    ds.take(lane, d, st);
    gam.get(g);
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i) {
      const F2 xh = mul2(x[i], rr);
      const F2 gy = mul2(d[i], g[i]);
      s2 = fma2(gy, xh, s2);
      if (GRADS && live) dg[i] = fma2(d[i], xh, dg[i]);
      d[i] = gy;
      x[i] = xh;
    }
    float s[1] = {sum2(s2)};
    row_sums<1, L>(s, group, sm[par]);
    par ^= 1;
    const float A = -rc * (s[0] * inv);
    const F2 AA = f2(A, A);
    if (RING) {
      F2 e[CPT / 2];
      es.take(lane, e, st);
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i) x[i] = fma2(d[i], rr, fma2(x[i], AA, e[i]));
    } else {
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i) x[i] = fma2(d[i], rr, mul2(x[i], AA));
    }
    if (++st == S) st = 0;
    if (live) {
      if (DH && !RING) add_row(lane, static_cast<const X*>(a.dh) + (int64_t)row * a.ld_dh, x);
      store_row(lane, dx, x);
    }
    dx += dx_step;
  }
  copy_wait<0>();
  if (!GRADS || !a.partial) return;
  // the block's column sums: its groups are added in order, the stores coalesced
  float* out = a.partial + (size_t)blockIdx.x * a.H;
  float* acc = reinterpret_cast<float*>(dyn) + (size_t)group * a.H;   // [ROWS][H]
  __syncthreads();                       // the ring is no longer read
#pragma unroll
  for (int i = 0; i < CPT / 2; ++i) {
    float gs[2];
    split(dg[i], gs[0], gs[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = (2 * i + k) / V, e = (2 * i + k) % V, c = lane.first() + j * L * V + e;
      if (SHIFT ? lane.inside(j, e) : lane.valid(j)) acc[c] = gs[k];
    }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(dyn);
  for (int c = threadIdx.x; c < a.H; c += TH) {
    float v = all[c];
#pragma unroll
    for (int g = 1; g < ROWS; ++g) v += all[(size_t)g * a.H + c];
    out[c] = v;
  }
}

// dgamma from the blocks' sums: 32 columns per block, 32 slices of the blocks,
// added as a fixed tree.
__global__ void __launch_bounds__(1024) rms_dgamma_kernel(const float* partial, int blocks, int H, int wtype,
                                                          void* dgamma) {
  __shared__ float sm[32][33];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H)
#pragma unroll 8
    for (int b = w; b < blocks; b += 32) v += partial[(size_t)b * H + c];
  sm[w][lane] = v;
  __syncthreads();
  const float s = lanes_sum<32>(sm[lane][w]);   // warp w sums column w of the tile
  const int cw = blockIdx.x * 32 + w;
  if (lane == 0 && cw < H) {
    if (wtype == MOE_TYPE_BF16) static_cast<__nv_bfloat16*>(dgamma)[cw] = __float2bfloat16_rn(s);
    else static_cast<float*>(dgamma)[cw] = s;
  }
}

// Rows that the kernel above does not take: dx with a block per row, two
// passes; the column sums from a read of their own, a thread per column.
template <typename X, int V>
__global__ void __launch_bounds__(1024) rms_bwd_rows_kernel(const RmsBwdArgs a) {
  __shared__ float sm[32];
  let_next_start();
  wait_for_previous();
  const int64_t row = blockIdx.x;
  const X* h = static_cast<const X*>(a.h) + row * a.ld_h;
  const X* dy = static_cast<const X*>(a.dy) + row * a.ld_dy;
  const X* dh = a.dh ? static_cast<const X*>(a.dh) + row * a.ld_dh : nullptr;
  const float r = a.rstd[row];
  float s[1] = {0.f};
#pragma unroll 4
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float d[V], v[V];
    load_part(dy + c, d);
    load_part(h + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] += d[i] * load_w1(a.gamma, a.wtype, c + i, 1.f) * (v[i] * r);
  }
  row_sums<1, 1024>(s, 0, sm);
  const float c2 = s[0] / (float)a.H;
  X* dx = static_cast<X*>(a.dx) + row * a.ld_dx;
#pragma unroll 2
  for (int c = threadIdx.x * V; c < a.H; c += 1024 * V) {
    float d[V], v[V], e[V] = {};
    load_part(dy + c, d);
    load_part(h + c, v);
    if (dh) load_part(dh + c, e);
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = r * (d[i] * load_w1(a.gamma, a.wtype, c + i, 1.f) - v[i] * r * c2) + e[i];
    store_part(dx + c, v);
  }
}

// (Runs before the kernel of dx, which may overwrite h, dy or dh.)
template <typename X>
__global__ void __launch_bounds__(256) rms_bwd_cols_kernel(const RmsBwdArgs a) {
  let_next_start();
  wait_for_previous();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float dg = 0.f;
#pragma unroll 8
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y)
    dg += to_f(static_cast<const X*>(a.dy)[row * a.ld_dy + c]) *
          (to_f(static_cast<const X*>(a.h)[row * a.ld_h + c]) * a.rstd[row]);
  a.partial[(size_t)blockIdx.y * a.H + c] = dg;
}

template <typename X>
cudaError_t backward_cols(const RmsBwdArgs& a, int64_t most, int* blocks, cudaStream_t s) {
  if (!a.partial) return cudaSuccess;
  const int64_t slabs = most < 64 ? most : 64;
  *blocks = (int)slabs;
  return launch_overlapped(rms_bwd_cols_kernel<X>, dim3((a.H + 255) / 256, (unsigned)slabs), 256, 0, s, a);
}

template <typename X, int V>
cudaError_t backward_rows(const RmsBwdArgs& a, int64_t most, int* blocks, cudaStream_t s) {
  const cudaError_t e = backward_cols<X>(a, most, blocks, s);
  if (e != cudaSuccess) return e;
  return launch_overlapped(rms_bwd_rows_kernel<X, V>, (unsigned)a.T, 1024, 0, s, a);
}

template <typename X, bool SHIFT, bool DH, int CPT, int L, int S, bool GRADS = true>
cudaError_t run_bwd(const RmsBwdArgs& a, const Offsets& o, int64_t most, int* blocks, cudaStream_t s) {
  static CtxCache<int> cache;
  constexpr int TH = kBlock<L, kThreads<X>>;
  constexpr int kRing = (DH && CPT <= 16 ? 3 : 2) * Stream<X, CPT, L, SHIFT, S, TH>::RING +
                        (CPT > 16 ? CPT * 4 * TH : 0);
  constexpr int kSums = kRows<L, kThreads<X>> * L * CPT * 4;    // H <= L CPT
  return run(rms_bwd_kernel<X, SHIFT, DH, CPT, L, S, GRADS>, cache, a, kRows<L, kThreads<X>>, TH,
             kRing > kSums ? kRing : kSums, SHIFT ? o.period : 1, most, blocks, s);
}

template <typename X, bool SHIFT, bool DH>
cudaError_t backward(const RmsBwdArgs& a, const Offsets& o, int64_t most, int* blocks, cudaStream_t s) {
  constexpr bool B = sizeof(X) == 2;
  constexpr int S = B ? 4 : 3;
  const int n = SHIFT ? a.H + kVec<X> - 1 : a.H;
  if (n <= 128) return run_bwd<X, SHIFT, DH, 8, 16, S>(a, o, most, blocks, s);
  if (n <= 512) return run_bwd<X, SHIFT, DH, 16, 32, S>(a, o, most, blocks, s);
  if (n <= 1024) return run_bwd<X, SHIFT, DH, 16, 64, S>(a, o, most, blocks, s);
  if (n <= 1536) return run_bwd<X, SHIFT, DH, 16, 96, S>(a, o, most, blocks, s);
  if (n <= 2048) return run_bwd<X, SHIFT, DH, 16, 128, S>(a, o, most, blocks, s);
  if (n <= 2560) return run_bwd<X, SHIFT, DH, 16, 160, S>(a, o, most, blocks, s);
  if (n <= 3584) return run_bwd<X, SHIFT, DH, 16, 224, S>(a, o, most, blocks, s);
  if (n <= 4096) return run_bwd<X, SHIFT, DH, 16, 256, S>(a, o, most, blocks, s);
  if (n <= 5632) return run_bwd<X, SHIFT, DH, 16, 352, 3>(a, o, most, blocks, s);
  if (n <= 8192) return run_bwd<X, SHIFT, DH, 16, 512, B ? 3 : 2>(a, o, most, blocks, s);
  if (n <= 16384) {
    if constexpr (B) {
      return run_bwd<X, SHIFT, DH, 32, 512, 2>(a, o, most, blocks, s);
    } else {   // the ring holds one row of both tensors, and the registers no sums
      const cudaError_t e = backward_cols<X>(a, most, blocks, s);
      if (e != cudaSuccess) return e;
      int unused;
      return run_bwd<X, SHIFT, DH, 32, 512, 1, false>(a, o, INT64_MAX, &unused, s);
    }
  }
  return backward_rows<X, SHIFT ? 1 : kVec<X>>(a, most, blocks, s);
}

template <typename X>
cudaError_t backward_any(const RmsBwdArgs& a, const Offsets& o, int64_t most, int* blocks, cudaStream_t s) {
  if (o.vectors)
    return a.dh ? backward<X, false, true>(a, o, most, blocks, s) : backward<X, false, false>(a, o, most, blocks, s);
  if (o.same)
    return a.dh ? backward<X, true, true>(a, o, most, blocks, s) : backward<X, true, false>(a, o, most, blocks, s);
  return backward_rows<X, 1>(a, most, blocks, s);
}

}  // namespace

cudaError_t launch_rms_norm_backward(const moe_rms_dims& d, const void* dy, const void* h, const void* dh,
                                     const void* gamma, const float* rstd, void* dx, void* dgamma, float* partial,
                                     cudaStream_t s) {
  const RmsBwdArgs a{dy, h, dh, gamma, rstd, dx, dgamma ? partial : nullptr, d.ld_y, d.ld_h, d.ld_dh, d.ld_dx,
                     d.T, d.H, d.w_type};
  const int es = d.x_type == MOE_TYPE_BF16 ? 2 : 4;
  int blocks = 0;
  if (d.T > 0) {
    const void* p[4] = {h, dy, dx, dh};
    const int64_t ld[4] = {d.ld_h, d.ld_y, d.ld_dx, d.ld_dh};
    const Offsets o = offsets_of(p, ld, dh ? 4 : 3, es, d.T, d.H);
    const int64_t most = norm_partial_blocks(d.T);
    const cudaError_t e = es == 2 ? backward_any<__nv_bfloat16>(a, o, most, &blocks, s)
                                  : backward_any<float>(a, o, most, &blocks, s);
    if (e != cudaSuccess) return e;
  }
  if (!dgamma) return cudaSuccess;
  return launch_overlapped(rms_dgamma_kernel, (d.H + 31) / 32, 1024, 0, s, (const float*)partial, blocks, d.H,
                           d.w_type, dgamma);
}

}  // namespace moe
