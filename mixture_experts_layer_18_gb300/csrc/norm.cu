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
#include "rows.cuh"

namespace moe {

namespace {

using namespace rows;

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
