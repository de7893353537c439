// clip.cu - global L2 norm of a list of gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2)
//   out  = g * (norm > max_norm ? max_norm / norm : 1)
//
// Bound by HBM: the norm reads every gradient once; clipping reads it again
// (the factor is known only after the last element) and writes it once.  The
// tensors are cut into chunks that blocks of one launch share out, whatever
// the tensors' number and sizes, so a list of many small tensors costs one
// launch per pass.  The list travels in the kernel's parameters: no table is
// copied to the device.
//
// A thread's squares are summed in fp32 over one chunk (at most 32 terms to an
// accumulator), everything above that in pairs of fp32 numbers (the sum and
// what its rounding lost, by Knuth's two-sum), which is about as exact as
// double: the GPU's double rate is so low that a block's sum and root in double
// took 5 us.  Chunks whose sum leaves the range in which fp32 keeps squares go
// through a double instead.  Every sum has a fixed order, so the norm is the
// same in every run on one GPU.
//
// Measured on 1.21 GB of bf16 gradients: the norm reads 6.4 TB/s.  The scaling
// pass wants every warp the SM can hold, each with two vectors on the way
// (32 warps with four each: 11% slower over both passes); the norm's pass does
// not care.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kNormPerSm = 4, kScalePerSm = 8;   // blocks per SM of the two passes
constexpr int kMaxBlocks = 1024;

// A launch's share of the list.
template <int N>
struct ClipList {
  const void* src[N];
  void* dst[N];
  int64_t n[N];
  int64_t first[N + 1];    // chunks before tensor i
  uint8_t type[N];
  int count;
  int chunk;               // elements per chunk (a multiple of 8)
};

template <int N>
__device__ __forceinline__ int tensor_of(const ClipList<N>& l, int64_t c) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A sum as hi + lo.
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float h, float l) {
    const float s = hi + h, t = s - hi;
    lo += ((hi - (s - t)) + (h - t)) + l;
    hi = s;
  }
};

// What a block hands on: its sum, and the part of it that was taken in double.
struct Partial {
  Sum2 sum;
  double wild;
};

// Sums over the block, the same in every thread.  The double one costs
// nothing where every thread's is zero.
__device__ __forceinline__ Partial block_sum(Partial v) {
  __shared__ Partial sm[kThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const bool wild = __syncthreads_or(v.wild != 0.0);     // (a NaN too)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, v.sum.hi, o), l = __shfl_xor_sync(0xffffffffu, v.sum.lo, o);
    v.sum.add(h, l);
    if (wild) v.wild += __shfl_xor_sync(0xffffffffu, v.wild, o);
  }
  if (lane == 0) sm[w] = v;
  __syncthreads();
  v = sm[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) {
    v.sum.add(sm[i].sum.hi, sm[i].sum.lo);
    if (wild) v.wild += sm[i].wild;
  }
  return v;
}

// ------------------------------------------------------------- elements
template <typename G>
struct Vec {
  static constexpr int N = 16 / sizeof(G);
};

template <typename G>
__device__ __forceinline__ float get(const G* p) {
  if constexpr (sizeof(G) == 2) return __bfloat162float(*p);
  else return *p;
}
template <typename G>
__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[Vec<G>::N]) {
  if constexpr (sizeof(G) == 2) {
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  } else {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  }
}

// Elements of [0, n) before the first 16-byte boundary.
template <typename G>
__device__ __forceinline__ int head_of(const G* p, int n) {
  const int h = (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(G);
  return h < n ? h : n;
}

// ----------------------------------------------------------------- norm
// Adds this thread's share of the squares of p[0, n).
template <typename G>
__device__ __forceinline__ void squares(const G* p, int n, Partial& acc) {
  constexpr int V = Vec<G>::N;
  const int head = head_of(p, n);
  const int nv = (n - head) / V;
  const uint4* pv = reinterpret_cast<const uint4*>(p + head);
  const int tail0 = head + nv * V;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t bits = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    const uint4 u = pv[i];
    bits |= (u.x | u.y) | (u.z | u.w);
    float v[V];
    unpack16<G>(u, v);
#pragma unroll
    for (int j = 0; j < V; ++j) s[j & 3] += v[j] * v[j];
  }
  if ((int)threadIdx.x < head) {
    const float v = get(p + threadIdx.x);
    bits |= __float_as_uint(v);
    s[0] += v * v;
  }
  if (tail0 + (int)threadIdx.x < n) {       // fewer than V elements are left
    const float v = get(p + tail0 + threadIdx.x);
    bits |= __float_as_uint(v);
    s[1] += v * v;
  }
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  // squares that left the range where fp32 keeps them (a sum beyond 2^80,
  // which leaves room for the sums of all chunks, or one below 2^-116, where a
  // square may have been rounded as a subnormal number) are taken again in
  // double; a NaN stays one
  const bool low = sum < 1.2e-35f && (bits & (sizeof(G) == 2 ? 0x7fff7fffu : 0x7fffffffu));
  if (!low && !(sum > 1.2e24f)) {
    acc.sum.add(sum, 0.f);
    return;
  }
  double d = 0.0;
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    float v[V];
    unpack16<G>(pv[i], v);
    for (int j = 0; j < V; ++j) d += (double)v[j] * (double)v[j];
  }
  if ((int)threadIdx.x < head) d += (double)get(p + threadIdx.x) * (double)get(p + threadIdx.x);
  if (tail0 + (int)threadIdx.x < n) {
    const double v = get(p + tail0 + threadIdx.x);
    d += v * v;
  }
  acc.wild += d;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kNormPerSm)
    grad_squares_kernel(const __grid_constant__ ClipList<N> l, Partial* partial) {
  let_next_start();
  wait_for_previous();
  Partial acc = {{0.f, 0.f}, 0.0};
  const int64_t chunks = l.first[l.count];
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(l, c);
    const int64_t e0 = (c - l.first[i]) * l.chunk;
    const int64_t left = l.n[i] - e0;
    const int n = left < l.chunk ? (int)left : l.chunk;
    if (l.type[i] == MOE_TYPE_BF16) squares(static_cast<const __nv_bfloat16*>(l.src[i]) + e0, n, acc);
    else squares(static_cast<const float*>(l.src[i]) + e0, n, acc);
  }
  acc = block_sum(acc);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// The norm from all blocks' partial sums (every thread gets it).
__device__ __forceinline__ float norm_of(const Partial* partial, int np) {
  Partial v = {{0.f, 0.f}, 0.0};
  for (int i = threadIdx.x; i < np; i += kThreads) {
    const Partial p = partial[i];
    v.sum.add(p.sum.hi, p.sum.lo);
    if (p.wild != 0.0) v.wild += p.wild;
  }
  v = block_sum(v);
  if (v.wild != 0.0) return (float)sqrt(v.wild + (double)v.sum.hi + (double)v.sum.lo);
  return sqrtf(v.sum.hi + v.sum.lo);
}

__device__ __forceinline__ void publish_norm(float norm, float* out, int32_t* status) {
  *out = norm;
  if (!(norm <= 3.402823466e38f)) report(status, MOE_ERR_BAD_INPUT);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const Partial* partial, int np, float* norm,
                                                             int32_t* status) {
  let_next_start();
  wait_for_previous();
  const float v = norm_of(partial, np);
  if (threadIdx.x == 0) publish_norm(v, norm, status);
}

// ----------------------------------------------------------------- clip
template <typename G>
__device__ __forceinline__ void scale_chunk(const G* p, G* q, int n, float c) {
  constexpr int V = Vec<G>::N;
  auto put = [&](int i) {
    const float v = get(p + i) * c;
    if constexpr (sizeof(G) == 2) q[i] = __float2bfloat16_rn(v);
    else q[i] = v;
  };
  // no common 16-byte boundary (200 M bf16 with the norm 456 us, else 203; fp32 573 and 381)
  if (((uintptr_t)p & 15) != ((uintptr_t)q & 15)) {
    for (int i = threadIdx.x; i < n; i += kThreads) put(i);
    return;
  }
  const int head = head_of(p, n);
  const int nv = (n - head) / V;
  const uint4* pv = reinterpret_cast<const uint4*>(p + head);
  uint4* qv = reinterpret_cast<uint4*>(q + head);
#pragma unroll 2
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    float v[V];
    unpack16<G>(pv[i], v);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= c;
    if constexpr (sizeof(G) == 2)
      qv[i] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                         pack_bf16(v[6], v[7]));
    else
      qv[i] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                         __float_as_uint(v[3]));
  }
  if ((int)threadIdx.x < head) put(threadIdx.x);
  if (head + nv * V + (int)threadIdx.x < n) put(head + nv * V + threadIdx.x);
}

// Every block adds the partial sums up itself (a few KB from L2), so no
// launch stands between the norm's pass and this one.  Chunks are taken from
// the end of the list: what the norm's pass read last is still in L2.
template <int N>
__global__ void __launch_bounds__(kThreads, kScalePerSm)
    grad_scale_kernel(const __grid_constant__ ClipList<N> l, const Partial* partial, int np,
                      float max_norm, float* norm, int32_t* status) {
  let_next_start();
  wait_for_previous();
  const float total = norm_of(partial, np);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) publish_norm(total, norm, status);
  // a norm that is not finite scales nothing (the status says so)
  const float c = total > max_norm && total <= 3.402823466e38f ? max_norm / total : 1.f;
  const int64_t chunks = l.first[l.count];
  for (int64_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const int64_t ck = chunks - 1 - k;
    const int i = tensor_of(l, ck);
    if (c == 1.f && l.src[i] == l.dst[i]) continue;
    const int64_t e0 = (ck - l.first[i]) * l.chunk;
    const int64_t left = l.n[i] - e0;
    const int n = left < l.chunk ? (int)left : l.chunk;
    if (l.type[i] == MOE_TYPE_BF16)
      scale_chunk(static_cast<const __nv_bfloat16*>(l.src[i]) + e0,
                  static_cast<__nv_bfloat16*>(l.dst[i]) + e0, n, c);
    else
      scale_chunk(static_cast<const float*>(l.src[i]) + e0, static_cast<float*>(l.dst[i]) + e0, n, c);
  }
}

// ------------------------------------------------------------------ host
// Elements per chunk: enough for every block to have several, between
// 2048 (a vector per thread) and 32768 elements.  (A dozen per block, for an
// evener share, measured 20% slower: a chunk starts with empty loads.)
int chunk_for(const moe_grad_tensor* t, int count, int blocks) {
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += t[i].n;
  int64_t c = total / (4 * (int64_t)blocks);
  c = c < 2048 ? 2048 : c > 32768 ? 32768 : c;
  return (int)(c / 2048 * 2048);
}

template <int N>
void fill(ClipList<N>& l, const moe_grad_tensor* t, int count, int chunk) {
  l.count = 0;
  l.chunk = chunk;
  l.first[0] = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const int k = l.count++;
    l.src[k] = t[i].src;
    l.dst[k] = t[i].dst;
    l.n[k] = t[i].n;
    l.type[k] = (uint8_t)t[i].type;
    l.first[k + 1] = l.first[k] + (t[i].n + chunk - 1) / chunk;
  }
}

int grid_of(int64_t chunks, int per_sm) {
  const int64_t b = (int64_t)sm_count() * per_sm;
  return (int)(chunks < b ? chunks : b);
}

template <int N>
cudaError_t run(const moe_grad_tensor* t, int count, bool clip, float max_norm, Partial* partial,
                float* norm, int32_t* status, cudaStream_t s) {
  const int chunk = chunk_for(t, count, sm_count() * kNormPerSm);
  ClipList<N> l;
  int np = 0;
  for (int i = 0; i < count; i += N) {
    fill(l, t + i, count - i < N ? count - i : N, chunk);
    if (l.count == 0) continue;
    int grid = grid_of(l.first[l.count], kNormPerSm);
    if (grid > kMaxBlocks) grid = kMaxBlocks;
    const cudaError_t e = launch_overlapped(grad_squares_kernel<N>, grid, kThreads, 0, s, l, partial + np);
    if (e != cudaSuccess) return e;
    np += grid;
  }
  bool told = false;
  if (clip)
    for (int i = (count - 1) / N * N; i >= 0 && count > 0; i -= N) {   // last launch's tensors first
      if (count > N) fill(l, t + i, count - i < N ? count - i : N, chunk);
      if (l.count == 0) continue;
      const cudaError_t e =
          launch_overlapped(grad_scale_kernel<N>, grid_of(l.first[l.count], kScalePerSm), kThreads, 0, s, l,
                       (const Partial*)partial, np, max_norm, told ? nullptr : norm, status);
      if (e != cudaSuccess) return e;
      told = true;
    }
  return told ? cudaSuccess
              : launch_overlapped(grad_norm_kernel, 1, kThreads, 0, s, (const Partial*)partial, np, norm, status);
}

constexpr int kShort = 48, kLong = 512;   // tensors per launch

}  // namespace

size_t grad_workspace_bytes(int count) {
  const int n = count <= kShort ? kShort : kLong;
  const size_t launches = count <= 0 ? 1 : ((size_t)count + n - 1) / n;
  return launches * kMaxBlocks * sizeof(Partial);
}

// Short lists use a small parameter block (a launch copies it).
cudaError_t launch_grad_clip(const moe_grad_tensor* t, int count, bool clip, float max_norm,
                             void* ws, float* norm, int32_t* status, cudaStream_t s) {
  Partial* partial = static_cast<Partial*>(ws);
  if (count <= kShort) return run<kShort>(t, count, clip, max_norm, partial, norm, status, s);
  return run<kLong>(t, count, clip, max_norm, partial, norm, status, s);
}

}  // namespace moe
