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
// from centred values, in a second sum: no cancellation), and the backward's
// column sums stay in registers over all rows of a block.  All sums are fp32
// trees in a fixed order; the results do not depend on timing.
//
// Lanes load 16-byte vectors where every row starts on a 16-byte boundary,
// single elements otherwise (odd widths or strides).
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kBwdThreads = 512;  // largest block of the fused backward

// ------------------------------------------------------------- elements
template <typename X, int VEC>
struct Raw {
  using type = uint4;
};
template <typename X>
struct Raw<X, 1> {
  using type = X;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename X, int VEC>
__device__ __forceinline__ void unpack(const typename Raw<X, VEC>::type& r, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = to_f(r);
  } else if constexpr (sizeof(X) == 2) {
    v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
    v[4] = bf16_lo(r.z); v[5] = bf16_hi(r.z); v[6] = bf16_lo(r.w); v[7] = bf16_hi(r.w);
  } else {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
  }
}

template <typename X, int VEC>
__device__ __forceinline__ void store_vec(X* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(X) == 2) *p = __float2bfloat16_rn(v[0]);
    else *p = v[0];
  } else if constexpr (sizeof(X) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// VEC weights from column c of a [H] vector of either type (NULL: `fill`).
template <int VEC>
__device__ __forceinline__ void load_w(const void* p, int type, int c, float fill, float (&v)[VEC]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = fill;
  } else if (type == MOE_TYPE_BF16) {
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p) + c;
    if constexpr (VEC == 8) {
      unpack<__nv_bfloat16, 8>(*reinterpret_cast<const uint4*>(w), v);
    } else if constexpr (VEC == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(w);
      v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = __bfloat162float(w[i]);
    }
  } else {
    const float* w = static_cast<const float*>(p) + c;
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(w + i);
        v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = w[i];
    }
  }
}

// ------------------------------------------------------------ reductions
// Sum over the L lanes of a row: a shuffle tree in the warp, then (L > 32)
// one named barrier per row group and a tree over its warps' sums.  `sm`
// holds one float per warp of the block and is not reused before the next
// barrier of the same group.
__device__ __forceinline__ void group_bar(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

__device__ __forceinline__ float lanes_sum(float v, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float row_sum(float v, int L, int group, float* sm) {
  v = lanes_sum(v, L < 32 ? L : 32);
  if (L <= 32) return v;
  const int warps = L >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sm[threadIdx.x >> 5] = v;
  group_bar(group, L);
  v = lane < warps ? sm[group * warps + lane] : 0.f;
  return lanes_sum(v, 32);
}

__device__ __forceinline__ float2 row_sum2(float2 v, int L, int group, float2* sm) {
  const int width = L < 32 ? L : 32;
  v.x = lanes_sum(v.x, width);
  v.y = lanes_sum(v.y, width);
  if (L <= 32) return v;
  const int warps = L >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sm[threadIdx.x >> 5] = v;
  group_bar(group, L);
  v = lane < warps ? sm[group * warps + lane] : make_float2(0.f, 0.f);
  v.x = lanes_sum(v.x, 32);
  v.y = lanes_sum(v.y, 32);
  return v;
}

// --------------------------------------------------------------- forward
struct FwdArgs {
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  int64_t ld_x, ld_y;
  int T, H, L, wtype;
  float eps;
};

// One row per group of L lanes, blockDim.x / L rows per block.
template <typename X, int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const FwdArgs a) {
  using R = typename Raw<X, VEC>::type;
  __shared__ float sm[2][32];
  const int L = a.L, group = threadIdx.x / L, t = threadIdx.x - group * L;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / L) + group;
  const bool live = row < a.T;
  const X* x = static_cast<const X*>(a.x) + (live ? row : 0) * a.ld_x;
  R raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * L + t) * VEC;
    if (live && c < a.H) raw[j] = *reinterpret_cast<const R*>(x + c);
  }
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (live && (j * L + t) * VEC < a.H) {
      float v[VEC];
      unpack<X, VEC>(raw[j], v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += v[i];
    }
  const float mu = row_sum(s, L, group, sm[0]) / (float)a.H;
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (live && (j * L + t) * VEC < a.H) {
      float v[VEC];
      unpack<X, VEC>(raw[j], v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) q += (v[i] - mu) * (v[i] - mu);
    }
  const float r = 1.f / sqrtf(row_sum(q, L, group, sm[1]) / (float)a.H + a.eps);
  if (!live) return;
  if (t == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  X* y = static_cast<X*>(a.y) + row * a.ld_y;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * L + t) * VEC;
    if (c < a.H) {
      float v[VEC], g[VEC], b[VEC];
      unpack<X, VEC>(raw[j], v);
      load_w<VEC>(a.gamma, a.wtype, c, 1.f, g);
      load_w<VEC>(a.beta, a.wtype, c, 0.f, b);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = (v[i] - mu) * r * g[i] + b[i];
      store_vec<X, VEC>(y + c, v);
    }
  }
}

// Rows longer than 1024 lanes x 32 columns: a block per row, three passes over it (the
// second and third find most of it in L2).
template <typename X>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const FwdArgs a) {
  __shared__ float sm[2][32];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  float s = 0.f;
  for (int c = threadIdx.x; c < a.H; c += 1024) s += to_f(x[c]);
  const float mu = row_sum(s, 1024, 0, sm[0]) / (float)a.H;
  float q = 0.f;
  for (int c = threadIdx.x; c < a.H; c += 1024) {
    const float d = to_f(x[c]) - mu;
    q += d * d;
  }
  const float r = 1.f / sqrtf(row_sum(q, 1024, 0, sm[1]) / (float)a.H + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = r;
  }
  X* y = static_cast<X*>(a.y) + row * a.ld_y;
  for (int c = threadIdx.x; c < a.H; c += 1024) {
    float g[1], b[1], v[1];
    load_w<1>(a.gamma, a.wtype, c, 1.f, g);
    load_w<1>(a.beta, a.wtype, c, 0.f, b);
    v[0] = (to_f(x[c]) - mu) * r * g[0] + b[0];
    store_vec<X, 1>(y + c, v);
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
  int T, H, L, wtype;
};

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Persistent blocks; each group of L lanes walks over rows with a stride of
// all groups of the grid.  With vectors, a lane's parts of the next S - 1
// rows of x and dy travel to its own slots of shared memory (asynchronous
// copies that only this lane reads, so no barrier orders them); with single
// elements the next row waits in registers.  The sums over a row take one
// barrier.
template <typename X, int VEC, int CPT, int S>
__global__ void __launch_bounds__(kBwdThreads, 1) norm_bwd_kernel(const BwdArgs a) {
  using R = typename Raw<X, VEC>::type;
  constexpr int NV = CPT / VEC;
  constexpr bool RING = VEC > 1;
  constexpr bool KEEP_G = CPT <= 16;    // gamma in registers, else re-read (L1)
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float2 sm[2][kBwdThreads / 32];
  const int L = a.L, group = threadIdx.x / L, t = threadIdx.x - group * L;
  const int R_ = blockDim.x / L;        // rows of a block in flight
  const int64_t stride = (int64_t)gridDim.x * R_;
  const X* xp = static_cast<const X*>(a.x);
  const X* dyp = static_cast<const X*>(a.dy);
  X* dxp = static_cast<X*>(a.dx);
  float gam[KEEP_G ? CPT : 1], dg[CPT], db[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) dg[i] = db[i] = 0.f;
  if constexpr (KEEP_G) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * L + t) * VEC;
      float g[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) g[i] = 0.f;
      if (c < a.H) load_w<VEC>(a.gamma, a.wtype, c, 1.f, g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) gam[j * VEC + i] = g[i];
    }
  }
  // ring slot of (stage, tensor, vector): one 16-byte word per thread
  const uint32_t ring0 = RING ? smem_u32(dyn) + threadIdx.x * 16 : 0;
  auto slot = [&](int st, int which, int j) -> uint32_t {
    return (uint32_t)(((st * 2 + which) * NV + j) * blockDim.x * 16);
  };
  auto fetch = [&](int64_t row, int st) {
    if (row < a.T) {
      const X* xr = xp + row * a.ld_x;
      const X* dr = dyp + row * a.ld_dy;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * L + t) * VEC;
        if (c < a.H) {
          copy16_async(ring0 + slot(st, 0, j), xr + c);
          copy16_async(ring0 + slot(st, 1, j), dr + c);
        }
      }
    }
    copy_commit();
  };
  R xn[RING ? 1 : NV], dn[RING ? 1 : NV];
  auto fetch_regs = [&](int64_t row) {
    if (row < a.T) {
      const X* xr = xp + row * a.ld_x;
      const X* dr = dyp + row * a.ld_dy;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * L + t) * VEC;
        if (c < a.H) {
          xn[j] = *reinterpret_cast<const R*>(xr + c);
          dn[j] = *reinterpret_cast<const R*>(dr + c);
        }
      }
    }
  };
  int64_t row = (int64_t)blockIdx.x * R_ + group;
  if constexpr (RING) {
#pragma unroll
    for (int st = 0; st < S - 1; ++st) fetch(row + st * stride, st);
  } else {
    fetch_regs(row);
  }
  float mu_n = 0.f, r_n = 0.f;
  if (row < a.T) {
    mu_n = a.mean[row];
    r_n = a.rstd[row];
  }
  int st = 0, par = 0;
  // every group of the block makes the same number of turns
  for (int64_t base = (int64_t)blockIdx.x * R_; base < a.T; base += stride, row += stride) {
    const bool live = row < a.T;
    const float mu = mu_n, r = r_n;
    if (row + stride < a.T) {
      mu_n = a.mean[row + stride];
      r_n = a.rstd[row + stride];
    }
    R xr[NV], dr[NV];
    if constexpr (RING) {
      fetch(row + (S - 1) * stride, st == 0 ? S - 1 : st - 1);
      copy_wait<S - 1>();
      const uint8_t* ring = dyn + threadIdx.x * 16;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        xr[j] = *reinterpret_cast<const R*>(ring + slot(st, 0, j));
        dr[j] = *reinterpret_cast<const R*>(ring + slot(st, 1, j));
      }
      if (++st == S) st = 0;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        xr[j] = xn[j];
        dr[j] = dn[j];
      }
      fetch_regs(row + stride);
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * L + t) * VEC;
      if (live && c < a.H) {
        float x[VEC], d[VEC], g[VEC];
        unpack<X, VEC>(xr[j], x);
        unpack<X, VEC>(dr[j], d);
        if constexpr (!KEEP_G) load_w<VEC>(a.gamma, a.wtype, c, 1.f, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float h = (x[i] - mu) * r;
          const float gy = d[i] * (KEEP_G ? gam[(j * VEC + i) % (KEEP_G ? CPT : 1)] : g[i]);
          s.x += gy;
          s.y += gy * h;
          dg[j * VEC + i] += d[i] * h;
          db[j * VEC + i] += d[i];
        }
      }
    }
    s = row_sum2(s, L, group, sm[par]);
    par ^= 1;
    const float c1 = s.x / (float)a.H, c2 = s.y / (float)a.H;
    if (live) {
      X* out = dxp + row * a.ld_dx;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * L + t) * VEC;
        if (c < a.H) {
          float x[VEC], d[VEC], g[VEC];
          unpack<X, VEC>(xr[j], x);
          unpack<X, VEC>(dr[j], d);
          if constexpr (!KEEP_G) load_w<VEC>(a.gamma, a.wtype, c, 1.f, g);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float h = (x[i] - mu) * r;
            const float gy = d[i] * (KEEP_G ? gam[(j * VEC + i) % (KEEP_G ? CPT : 1)] : g[i]);
            x[i] = r * (gy - c1 - h * c2);
          }
          store_vec<X, VEC>(out + c, x);
        }
      }
    }
  }
  if (!a.partial) return;
  // the block's column sums: groups of one block are added in order
  float* out = a.partial + (size_t)blockIdx.x * 2 * a.H;
  if constexpr (RING) copy_wait<0>();
  if (R_ == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * L + t) * VEC;
      if (c < a.H)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          out[c + i] = dg[j * VEC + i];
          out[a.H + c + i] = db[j * VEC + i];
        }
    }
    return;
  }
  __syncthreads();                       // the ring is no longer read
  float* acc = reinterpret_cast<float*>(dyn);   // [R_][2][H]
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * L + t) * VEC;
    if (c < a.H)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        acc[(size_t)(2 * group) * a.H + c + i] = dg[j * VEC + i];
        acc[(size_t)(2 * group + 1) * a.H + c + i] = db[j * VEC + i];
      }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.H; c += blockDim.x) {
    float v = 0.f;
    for (int g = 0; g < R_; ++g) v += acc[(size_t)2 * g * a.H + c];
    out[c] = v;
  }
}

// dgamma and dbeta from the blocks' partial sums: 32 columns per block, 32
// slices of the partials, added as a fixed tree.
__global__ void __launch_bounds__(1024) norm_param_grad_kernel(const float* partial, int blocks, int H,
                                                               int wtype, void* dgamma, void* dbeta) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H)
    for (int b = w; b < blocks; b += 32) v += partial[((size_t)b * 2 + blockIdx.y) * H + c];
  sm[w][lane] = v;
  __syncthreads();
  const float s = lanes_sum(sm[lane][w], 32);   // warp w sums column w of the tile
  const int cw = blockIdx.x * 32 + w;
  void* out = blockIdx.y ? dbeta : dgamma;
  if (lane == 0 && cw < H && out) {
    if (wtype == MOE_TYPE_BF16) static_cast<__nv_bfloat16*>(out)[cw] = __float2bfloat16_rn(s);
    else static_cast<float*>(out)[cw] = s;
  }
}

// Rows that the fused kernel cannot hold: dx with a block per row (two
// passes), the column sums from a second read with a thread per column.
template <typename X>
__global__ void __launch_bounds__(1024) norm_bwd_rows_long_kernel(const BwdArgs a) {
  __shared__ float2 sm[32];
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  const X* dy = static_cast<const X*>(a.dy) + row * a.ld_dy;
  const float mu = a.mean[row], r = a.rstd[row];
  float2 s = make_float2(0.f, 0.f);
  for (int c = threadIdx.x; c < a.H; c += 1024) {
    float g[1];
    load_w<1>(a.gamma, a.wtype, c, 1.f, g);
    const float gy = to_f(dy[c]) * g[0];
    s.x += gy;
    s.y += gy * ((to_f(x[c]) - mu) * r);
  }
  s = row_sum2(s, 1024, 0, sm);
  const float c1 = s.x / (float)a.H, c2 = s.y / (float)a.H;
  X* dx = static_cast<X*>(a.dx) + row * a.ld_dx;
  for (int c = threadIdx.x; c < a.H; c += 1024) {
    float g[1], v[1];
    load_w<1>(a.gamma, a.wtype, c, 1.f, g);
    v[0] = r * (to_f(dy[c]) * g[0] - c1 - (to_f(x[c]) - mu) * r * c2);
    store_vec<X, 1>(dx + c, v);
  }
}

template <typename X>
__global__ void __launch_bounds__(256) norm_bwd_cols_long_kernel(const BwdArgs a) {
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
int ceil_pow2(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// Lanes per row so that a lane has at most `cpt` columns: a power of two up
// to a warp, then whole warps.
int lanes_for(int H, int cpt) {
  const int need = (H + cpt - 1) / cpt;
  return need <= 32 ? ceil_pow2(need) : (need + 31) / 32 * 32;
}

template <typename X, int VEC, int NV>
cudaError_t run_fwd(FwdArgs& a, int L, cudaStream_t s) {
  a.L = L;
  const int rows = L >= 256 ? 1 : 256 / L;
  const int64_t blocks = ((int64_t)a.T + rows - 1) / rows;
  norm_fwd_kernel<X, VEC, NV><<<(unsigned)blocks, rows * L, 0, s>>>(a);
  return cudaGetLastError();
}

// A lane takes up to 32 columns (fp32 vectors: 16, or 32 in rows over 16384)
// when there are rows enough to fill the GPU, else fewer, so that a few rows
// spread over more lanes.
template <typename X, int VEC>
cudaError_t fwd_typed(FwdArgs& a, cudaStream_t s) {
  constexpr int V = VEC == 1 ? 1 : VEC;
  const int64_t few = (int64_t)a.T * a.H;
  for (int cpt : {8, 16, 32}) {
    if (cpt < V) continue;
    const int L = lanes_for(a.H, cpt);
    if (L > 1024) continue;
    // spread a small problem; otherwise the widest share that fits
    const bool small = few <= (int64_t)sm_count() * 1024 * cpt;
    if (!small && cpt < (sizeof(X) == 4 ? 16 : 32) && lanes_for(a.H, cpt * 2) >= 32) continue;
    if constexpr (VEC == 1) {
      switch (cpt) {
        case 8: return run_fwd<X, 1, 8>(a, L, s);
        case 16: return run_fwd<X, 1, 16>(a, L, s);
        case 32: return run_fwd<X, 1, 32>(a, L, s);
      }
    } else {
      switch (cpt) {
        case 8: return run_fwd<X, VEC, 8 / VEC>(a, L, s);
        case 16: return run_fwd<X, VEC, 16 / VEC>(a, L, s);
        case 32: return run_fwd<X, VEC, 32 / VEC>(a, L, s);
      }
    }
  }
  norm_fwd_long_kernel<X><<<(unsigned)a.T, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

// Resident blocks per SM of one form of the backward, by warps per block.
struct Occupancy {
  int per_sm[kBwdThreads / 32 + 1];
};

template <typename X, int VEC, int CPT, int S>
cudaError_t run_bwd(BwdArgs& a, int64_t max_blocks, int* blocks_out, cudaStream_t s) {
  auto kern = norm_bwd_kernel<X, VEC, CPT, S>;
  const int L = lanes_for(a.H, CPT);
  a.L = L;
  const int rows = L >= 256 ? 1 : 256 / L;
  const int threads = rows * L;
  constexpr int kRing = VEC > 1 ? S * 2 * (CPT / VEC) * 16 : 0;    // bytes per thread
  const int sums = rows > 1 ? rows * 2 * a.H * 4 : 0;
  const int smem = kRing * threads > sums ? kRing * threads : sums;
  static CtxCache<Occupancy> cache;
  Occupancy occ;
  cudaError_t e = cache.get(&occ, [&](Occupancy* o) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kRing * kBwdThreads > 65536 ? kRing * kBwdThreads : 65536);
    o->per_sm[0] = 1;
    for (int w = 1; w <= kBwdThreads / 32 && r == cudaSuccess; ++w)
      r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o->per_sm[w], kern, 32 * w, kRing * 32 * w);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int per_sm = occ.per_sm[threads / 32];
  int64_t blocks = (int64_t)sm_count() * (per_sm < 1 ? 1 : per_sm);
  const int64_t need = ((int64_t)a.T + rows - 1) / rows;
  if (blocks > need) blocks = need;
  if (blocks > max_blocks) blocks = max_blocks;
  kern<<<(unsigned)blocks, threads, smem, s>>>(a);
  *blocks_out = (int)blocks;
  return cudaGetLastError();
}

// The fused kernel holds rows of up to 512 lanes x 16 columns (bf16 vectors:
// 32 columns); longer ones take the two-kernel form.
template <typename X, int VEC>
cudaError_t bwd_typed(BwdArgs& a, int64_t max_blocks, int* blocks, cudaStream_t s) {
  constexpr int ES = sizeof(X);
  if constexpr (VEC > 1) {
    if (lanes_for(a.H, 8) <= 32) return run_bwd<X, VEC, 8, 4>(a, max_blocks, blocks, s);
    if (lanes_for(a.H, 16) <= kBwdThreads)
      return run_bwd<X, VEC, 16, (ES == 2 ? 4 : 3)>(a, max_blocks, blocks, s);
    if constexpr (ES == 2)
      if (lanes_for(a.H, 32) <= kBwdThreads) return run_bwd<X, VEC, 32, 3>(a, max_blocks, blocks, s);
  } else {
    if (lanes_for(a.H, 8) <= kBwdThreads) return run_bwd<X, 1, 8, 1>(a, max_blocks, blocks, s);
    if (lanes_for(a.H, 16) <= kBwdThreads) return run_bwd<X, 1, 16, 1>(a, max_blocks, blocks, s);
  }
  norm_bwd_rows_long_kernel<X><<<(unsigned)a.T, 1024, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  int64_t slabs = 64;
  if (slabs > a.T) slabs = a.T;
  if (slabs > max_blocks) slabs = max_blocks;
  norm_bwd_cols_long_kernel<X><<<dim3((a.H + 255) / 256, (unsigned)slabs), 256, 0, s>>>(a);
  *blocks = (int)slabs;
  return cudaGetLastError();
}

bool rows16(const void* p, int64_t ld, int es) {
  return ((uintptr_t)p & 15) == 0 && (ld * es) % 16 == 0;
}

}  // namespace

cudaError_t launch_layer_norm(const NormDesc& d, const void* x, const void* gamma, const void* beta,
                              void* y, float* mean, float* rstd, cudaStream_t s) {
  FwdArgs a{x, gamma, beta, y, mean, rstd, d.ld_x, d.ld_y, d.T, d.H, 0, d.wtype, d.eps};
  const int es = d.xtype == MOE_TYPE_BF16 ? 2 : 4;
  const bool vec = (d.H * es) % 16 == 0 && rows16(x, d.ld_x, es) && rows16(y, d.ld_y, es) &&
                   ((uintptr_t)gamma & 15) == 0 && ((uintptr_t)beta & 15) == 0;
  if (es == 2) return vec ? fwd_typed<__nv_bfloat16, 8>(a, s) : fwd_typed<__nv_bfloat16, 1>(a, s);
  return vec ? fwd_typed<float, 4>(a, s) : fwd_typed<float, 1>(a, s);
}

int64_t norm_partial_blocks(int T) { return T < 1024 ? T : 1024; }

cudaError_t launch_layer_norm_backward(const NormDesc& d, const void* dy, const void* x,
                                       const void* gamma, const float* mean, const float* rstd,
                                       void* dx, void* dgamma, void* dbeta, float* partial,
                                       cudaStream_t s) {
  const bool params = dgamma || dbeta;
  BwdArgs a{dy, x, gamma, mean, rstd, dx, params ? partial : nullptr, d.ld_y, d.ld_x, d.ld_dx,
            d.T, d.H, 0, d.wtype};
  const int es = d.xtype == MOE_TYPE_BF16 ? 2 : 4;
  int blocks = 0;
  if (d.T > 0) {
    const bool vec = (d.H * es) % 16 == 0 && rows16(x, d.ld_x, es) && rows16(dy, d.ld_y, es) &&
                     rows16(dx, d.ld_dx, es) && ((uintptr_t)gamma & 15) == 0;
    const int64_t most = norm_partial_blocks(d.T);
    cudaError_t e;
    if (es == 2)
      e = vec ? bwd_typed<__nv_bfloat16, 8>(a, most, &blocks, s)
              : bwd_typed<__nv_bfloat16, 1>(a, most, &blocks, s);
    else
      e = vec ? bwd_typed<float, 4>(a, most, &blocks, s) : bwd_typed<float, 1>(a, most, &blocks, s);
    if (e != cudaSuccess) return e;
  }
  if (params) {
    norm_param_grad_kernel<<<dim3((d.H + 31) / 32, 2), 1024, 0, s>>>(partial, blocks, d.H, d.wtype,
                                                                   dgamma, dbeta);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace moe
