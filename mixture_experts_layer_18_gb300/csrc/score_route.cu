// score_route.cu - routing by scores: softmax or sigmoid scores, a bias for
// balance, groups of experts, top-k, gates; its backward; the bias' update.
//
//   s = softmax(l) or 1 / (1 + exp(-l)),  u = s + bias
//   a group's value is the sum of its `group_top` largest u; the `top_groups`
//   best groups stay; the k largest u in them are chosen (ties: the lower
//   index), and gate_j = scale s_j, or scale s_j / sum of the chosen s.
//
// The choice is that of u in 64 bits, whatever the GPU: values are computed in
// fp32 and compared, and a token in which two values that a comparison decides
// between lie within the error of fp32 (kNear) is done again in 64 bits by its
// warp.  (About one token in a thousand with 256 sigmoid scores; fp64 for all
// would take 30 times the time that the logits take from HBM.)  Without a bias
// u orders as the logits do, which are compared themselves.
//
// One warp per token, C neighbouring experts per lane, so that a group is a
// segment of lanes and the logits arrive in vectors.
#include "rows.cuh"

namespace moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;

using rows::put;
using rows::to_f;

// Total order of fp32 numbers (no NaN) as unsigned ones; 0 lies below -inf and
// stands for an expert that is absent, taken or in a group that went.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);        // (-0 becomes 0)
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// exp(x) by one MUFU instruction: relative error below 2^-22 + |x| 2^-23.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504088896341f));
  return r;
}

struct ScoreArgs {
  const void* logits;
  const float* bias;
  int64_t ld;
  int T, E, k, per_block;
  int groups, group_size, top_groups, group_top;
  int sigmoid, renorm;
  float scale;
  int32_t* idx;
  float* gate;
  int32_t* hist;            // [blocks][E]
  int32_t* status;
};

// A logit as it counts: NaN and +inf have no score; they read as -inf, which
// is a masked expert.
template <typename X>
__device__ __forceinline__ float logit(const ScoreArgs& a, const X* row, int e, bool* bad) {
  const float v = to_f(row[e]);
  if (v < INFINITY) return v;
  *bad = true;
  return -INFINITY;
}
__device__ __forceinline__ float bias_of(const ScoreArgs& a, int e) {
  const float b = a.bias ? a.bias[e] : 0.f;
  return fabsf(b) < INFINITY ? b : 0.f;
}

// The choice for one token in 64 bits; lane j < k gets the j-th expert.
template <typename X, int C>
__device__ __noinline__ int choose64(const ScoreArgs& a, const X* row) {
  const int lane = threadIdx.x & 31;
  double u[C];
  uint32_t out = 0;                       // absent, taken or gone
  bool bad = false;
  double top = -INFINITY, sum = 0;
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const int e = lane * C + q;
    u[q] = e < a.E ? (double)logit(a, row, e, &bad) : -INFINITY;
    if (e >= a.E) out |= 1u << q;
    top = fmax(top, u[q]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const bool masked = !(u[q] > -INFINITY);
    if (a.sigmoid) u[q] = 1.0 / (1.0 + exp(-u[q]));
    else u[q] = masked ? 0.0 : exp(u[q] - top);
    sum += u[q];
    if (masked) u[q] = -INFINITY;
  }
  sum = a.sigmoid ? 1.0 : warp_sum(sum);
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const int e = lane * C + q;
    if (e < a.E && u[q] > -INFINITY) u[q] = u[q] / sum + (double)bias_of(a, e);
  }
  if (a.groups > 1) {
    double mine = -INFINITY;              // lane i: the value of group i
    for (int g = 0; g < a.groups; ++g) {
      double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const int e = lane * C + q;
        if (e >= g * a.group_size && e < (g + 1) * a.group_size) {
          m2 = fmax(m2, fmin(m1, u[q]));
          m1 = fmax(m1, u[q]);
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const double n1 = __shfl_xor_sync(kAll, m1, o), n2 = __shfl_xor_sync(kAll, m2, o);
        m2 = fmax(fmin(m1, n1), fmax(m2, n2));
        m1 = fmax(m1, n1);
      }
      if (lane == g) mine = a.group_top == 1 ? m1 : m1 + m2;
    }
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double v = __shfl_sync(kAll, mine, g);
      better += v > mine || (v == mine && g < lane);
    }
    const unsigned stay = __ballot_sync(kAll, lane < a.groups && better < a.top_groups);
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int e = lane * C + q;
      if (e < a.E && !(stay >> (e / a.group_size) & 1u)) out |= 1u << q;
    }
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int be = kMaxE;
#pragma unroll
    for (int q = C - 1; q >= 0; --q)
      if (!(out >> q & 1u) && u[q] >= bv) {
        bv = u[q];
        be = lane * C + q;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double ov = __shfl_xor_sync(kAll, bv, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      if (ov > bv || (ov == bv && oe < be)) {
        bv = ov;
        be = oe;
      }
    }
    if (be / C == lane) out |= 1u << (be % C);
    if (lane == j) mine = be;
  }
  return mine;
}

// Largest distance of two fp32 values u that may be in the other order (or
// equal) in 64 bits.  Sigmoid: fast_exp's error enters as s (1 - s) (2^-22 +
// |l| 2^-23), at most 2^-24 + 2^-25; the sum, the reciprocal and the bias round
// by 2^-24, 2^-23 and 2^-24 |u|: below 2^-22 (1 + |u|) each, 2^-21 a pair, taken
// twice.  Softmax: as much relative to the largest score, and the sum's own
// relative error (fast_exp's, and C + 5 additions): below 2^-19.
__device__ __forceinline__ float near_of(bool sigmoid, float largest_s, float u) {
  return (sigmoid ? 0x1p-20f : 0x1p-18f * largest_s) + 0x1p-20f * fabsf(u);
}

template <typename X, int C, bool GROUPED>
__global__ void __launch_bounds__(1024) score_route_kernel(const __grid_constant__ ScoreArgs a) {
  __shared__ int hist[kMaxE];
  let_next_start();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.per_block;
  const int64_t t1 = min((int64_t)a.T, t0 + a.per_block);
  const bool by_logit = !a.bias && (!GROUPED || a.group_top == 1);
  float bias[C];
  bool bad = false;
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const int e = lane * C + q;
    bias[q] = e < a.E ? bias_of(a, e) : 0.f;
    if (a.bias && e < a.E && !(fabsf(a.bias[e]) < INFINITY)) bad = true;
  }
  for (int64_t t = t0 + (threadIdx.x >> 5); t < t1; t += blockDim.x >> 5) {
    const X* row = static_cast<const X*>(a.logits) + t * a.ld;
    float u[C];
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int e = lane * C + q;
      u[q] = e < a.E ? logit(a, row, e, &bad) : -INFINITY;
    }
    // the softmax' largest logit and sum
    float top = 0.f, sum = 1.f;
    if (!a.sigmoid && (!by_logit || !a.renorm)) {
      top = u[0];
#pragma unroll
      for (int q = 1; q < C; ++q) top = fmaxf(top, u[q]);
      top = warp_max(top);
      top = top > -INFINITY ? top : 0.f;
      sum = 0.f;
#pragma unroll
      for (int q = 0; q < C; ++q) sum += fast_exp(u[q] - top);
      sum = warp_sum(sum);
    }
    uint32_t key[C];
    if (by_logit) {
#pragma unroll
      for (int q = 0; q < C; ++q) key[q] = key_of(u[q]);
    } else {
      const float inv = 1.f / sum;
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const float s = a.sigmoid ? __fdividef(1.f, 1.f + fast_exp(-u[q])) : fast_exp(u[q] - top) * inv;
        key[q] = key_of(u[q] > -INFINITY ? s + bias[q] : -INFINITY);
      }
    }
#pragma unroll
    for (int q = 0; q < C; ++q)
      if (lane * C + q >= a.E) key[q] = 0;
    bool again = false;
    if (GROUPED) {
      float mine = -INFINITY;              // lane i: the value of group i
      for (int g = 0; g < a.groups; ++g) {
        uint32_t m1 = 0, m2 = 0;
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const int e = lane * C + q;
          if (e >= g * a.group_size && e < (g + 1) * a.group_size) {
            m2 = max(m2, min(m1, key[q]));
            m1 = max(m1, key[q]);
          }
        }
        const uint32_t best = __reduce_max_sync(kAll, m1);
        float v = value_of(best);
        if (a.group_top > 1) {
          const unsigned who = __ballot_sync(kAll, m1 == best);
          v += value_of(__reduce_max_sync(kAll, lane == __ffs(who) - 1 ? m2 : m1));
        }
        if (lane == g) mine = v;
      }
      int better = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float v = __shfl_sync(kAll, mine, g);
        better += v > mine || (v == mine && g < lane);
      }
      const bool stays = lane < a.groups && better < a.top_groups;
      const unsigned stay = __ballot_sync(kAll, stays);
      if (!by_logit && a.top_groups < a.groups) {
        const float lo = -warp_max(stays ? -mine : -INFINITY);
        const float hi = warp_max(lane < a.groups && !stays ? mine : -INFINITY);
        again = hi > -INFINITY && !(lo - hi > 2.f * near_of(a.sigmoid, 1.f / sum, fmaxf(fabsf(lo), fabsf(hi))));
      }
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const int e = lane * C + q;
        if (e < a.E && !(stay >> (e / a.group_size) & 1u)) key[q] = 0;
      }
    }
    // k rounds of a warp maximum, and one more for the value that just missed
    uint32_t sel = 0;
    int sel_e = 0;
    const int rounds = a.k + (by_logit || a.k == 32 ? 0 : 1);
    for (int j = 0; j < rounds; ++j) {
      uint32_t m = key[0];
#pragma unroll
      for (int q = 1; q < C; ++q) m = max(m, key[q]);
      const uint32_t best = __reduce_max_sync(kAll, m);
      const int who = __ffs(__ballot_sync(kAll, m == best)) - 1;
      int at = 0;
      if (lane == who) {
        bool open = true;
#pragma unroll
        for (int q = 0; q < C; ++q)
          if (open && key[q] == best) {
            key[q] = 0;
            at = q;
            open = false;
          }
      }
      at = __shfl_sync(kAll, at, who);
      if (lane == j) {
        sel = best;
        sel_e = who * C + at;
      }
    }
    float l = -INFINITY;
    bool unused = false;
    if (lane < rounds && sel) l = logit(a, row, sel_e, &unused);
    if (!by_logit) {
      const float v = sel ? value_of(sel) : -INFINITY, b = sel ? bias_of(a, sel_e) : 0.f;
      const float pv = __shfl_up_sync(kAll, v, 1), pl = __shfl_up_sync(kAll, l, 1), pb = __shfl_up_sync(kAll, b, 1);
      const bool close = lane > 0 && lane < rounds && v > -INFINITY && !(pl == l && pb == b) &&
                         !(pv - v > near_of(a.sigmoid, 1.f / sum, fmaxf(fabsf(pv), fabsf(v))));
      again = again || __any_sync(kAll, close) || a.k == 32;
      if (again) {
        sel_e = choose64<X, C>(a, row);
        if (lane < a.k) l = logit(a, row, sel_e, &unused);
      }
    }
    if (lane >= a.k) l = -INFINITY;
    // gates, relative to the largest chosen score where they are renormalised
    const bool none = !__any_sync(kAll, l > -INFINITY);
    float w;
    if (a.renorm) {
      const float x = a.sigmoid ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;      // log s (+ a constant)
      const float m = warp_max(x);
      w = l > -INFINITY ? expf(x - m) : 0.f;
      w = w / warp_sum(w);
    } else {
      w = !(l > -INFINITY) ? 0.f : a.sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - top) / sum;
    }
    if (none) bad = true;
    if (lane < a.k) {
      a.idx[t * a.k + lane] = sel_e;
      a.gate[t * a.k + lane] = none ? 0.f : a.scale * w;
      atomicAdd(&hist[sel_e], 1);
    }
  }
  if (bad) report(a.status, MOE_ERR_BAD_INPUT);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// ---------------------------------------------------------- permutation
struct PlaceArgs {
  const int32_t* idx;
  const int32_t* hist;       // [nb][E]
  int n_assign, E, nb, per_block;      // per_block: assignments of one router block
  int64_t max_rows;
  int32_t* counts;
  int32_t* offsets;
  int32_t* padded;
  int32_t* row_of;
  int32_t* assign_of;
  int32_t* status;
};

// Exclusive sum over the block's threads; `sm` has 33 ints.  *total: the sum.
__device__ __forceinline__ int block_scan(int v, int* sm, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sm[w] = x;
  __syncthreads();
  if (w == 0) {
    int y = lane < nw ? sm[lane] : 0;
    const int own = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(kAll, y, o);
      if (lane >= o) y += z;
    }
    sm[lane] = y - own;
    if (lane == 31) sm[32] = y;
  }
  __syncthreads();
  *total = sm[32];
  return sm[w] + x - v;
}

// Blocks [0, nb): rows of this block's assignments.  Every block adds the
// router's histograms up by itself (their sum over all blocks gives the rows'
// start of each expert, that over the blocks before it its own share), which
// saves a launch between the two.  Blocks from nb on: the rows without an assignment.
__global__ void __launch_bounds__(1024) place_kernel(const __grid_constant__ PlaceArgs a) {
  __shared__ int run[kMaxE], cnt[kMaxE], start[kMaxE + 1], sm[33];
  extern __shared__ uint16_t warps[];      // [32][E]
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int b = blockIdx.x;
  int total = 0, before = 0;
  if ((int)threadIdx.x < a.E) {
#pragma unroll 8
    for (int i = 0; i < a.nb; ++i) {
      const int c = a.hist[(int64_t)i * a.E + threadIdx.x];
      total += c;
      before += i < b ? c : 0;
    }
  }
  int rows, all;
  const int padded = (total + kAlign - 1) / kAlign * kAlign;
  const int first = block_scan(padded, sm, &rows);
  const int off = block_scan(total, sm, &all);
  if ((int)threadIdx.x < a.E) {
    run[threadIdx.x] = first + before;
    cnt[threadIdx.x] = total;
    start[threadIdx.x] = first;
    if (b == 0) {
      a.counts[threadIdx.x] = total;
      a.offsets[threadIdx.x] = off;
      a.padded[threadIdx.x] = first;
    }
  }
  if (threadIdx.x == 0) {
    start[a.E] = rows;
    if (b == 0) {
      a.offsets[a.E] = all;
      a.padded[a.E] = rows;
    }
  }
  __syncthreads();
  if (b >= a.nb) {
    const int pb = b - a.nb, npb = gridDim.x - a.nb;
    for (int e = pb * 32 + w; e < a.E; e += npb * 32)
      for (int r = start[e] + cnt[e] + lane; r < start[e + 1]; r += 32) a.assign_of[r] = -1;
    for (int64_t r = rows + (int64_t)pb * 1024 + threadIdx.x; r < a.max_rows; r += (int64_t)npb * 1024)
      a.assign_of[r] = -1;
    return;
  }
  const int64_t a0 = (int64_t)b * a.per_block, a1 = min((int64_t)a.n_assign, a0 + a.per_block);
  for (int64_t base = a0; base < a1; base += 1024) {
    // ranks within a warp by lane, of warps by their number, so that an
    // expert's rows follow the order of the assignments
    for (int i = threadIdx.x; i < 32 * a.E; i += 1024) warps[i] = 0;
    __syncthreads();
    const int64_t i = base + threadIdx.x;
    const int e = i < a1 ? a.idx[i] : -1;
    const unsigned same = __match_any_sync(kAll, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) warps[w * a.E + e] = (uint16_t)__popc(same);
    __syncthreads();
    if ((int)threadIdx.x < a.E) {
      int at = 0;
#pragma unroll 8
      for (int v = 0; v < 32; ++v) {
        const int c = warps[v * a.E + threadIdx.x];
        warps[v * a.E + threadIdx.x] = (uint16_t)at;
        at += c;
      }
      cnt[threadIdx.x] = run[threadIdx.x];
      run[threadIdx.x] += at;
    }
    __syncthreads();
    if (e >= 0) {
      const int row = cnt[e] + warps[w * a.E + e] + rank;
      a.row_of[i] = row;
      a.assign_of[row] = (int)i;
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------- backward
struct ScoreBwdArgs {
  const void* logits;
  const int32_t* idx;
  const float* gate;
  const float* dgate;
  void* dlogits;
  int64_t ld;
  int T, E, k, sigmoid, renorm;
  float scale;
  int32_t* status;
};

// One warp per token: the row is written once (zeros, or the softmax' share of
// all experts), then the chosen experts' elements.
template <typename X>
__global__ void __launch_bounds__(256) score_route_backward_kernel(const __grid_constant__ ScoreBwdArgs a) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * 8;
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < a.T; t += step) {
    const X* row = static_cast<const X*>(a.logits) + t * a.ld;
    X* out = static_cast<X*>(a.dlogits) + t * a.E;
    int e = -1;
    float w = 0.f, dw = 0.f;
    if (lane < a.k) {
      e = a.idx[t * a.k + lane];
      w = a.gate[t * a.k + lane];
      dw = a.dgate[t * a.k + lane];
      if (e < 0 || e >= a.E) {
        report(a.status, MOE_ERR_BAD_INDEX);
        e = -1;
      }
    }
    const float inner = warp_sum(w * dw);
    float d;
    if (a.sigmoid || a.renorm) {
      d = a.renorm ? w * (dw - inner / a.scale) : w * dw;
      if (a.sigmoid && e >= 0) d *= 1.f / (1.f + expf(to_f(row[e])));      // 1 - s
      for (int c = lane; c < a.E; c += 32) put(out + c, 0.f);
    } else {
      float top = -INFINITY, sum = 0.f;
      for (int c = lane; c < a.E; c += 32) {
        const float v = to_f(row[c]);
        if (v < INFINITY) top = fmaxf(top, v);
      }
      top = warp_max(top);
      if (!(top > -INFINITY)) top = 0.f;
      for (int c = lane; c < a.E; c += 32) {
        const float v = to_f(row[c]);
        if (v < INFINITY) sum += expf(v - top);
      }
      const float f = inner / fmaxf(warp_sum(sum), 1e-30f);
      for (int c = lane; c < a.E; c += 32) {
        const float v = to_f(row[c]);
        put(out + c, v < INFINITY ? -f * expf(v - top) : 0.f);
      }
      d = w * dw;
      if (e >= 0) {
        const float v = to_f(row[e]);
        if (v < INFINITY) d -= f * expf(v - top);
      }
    }
    __syncwarp();
    if (e >= 0) put(out + e, d);
  }
}

__global__ void __launch_bounds__(256) balance_bias_kernel(const int32_t* counts, int E, float rate, const float* bias,
                                                           float* out) {
  __shared__ long long part[8];
  let_next_start();
  wait_for_previous();
  long long n = 0;
  for (int e = threadIdx.x; e < E; e += 256) n += counts[e];
  n = warp_sum(n);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) n += part[i];
  for (int e = threadIdx.x; e < E; e += 256) {
    const long long c = (long long)counts[e] * E;
    out[e] = bias[e] + (c < n ? rate : c > n ? -rate : 0.f);
  }
}

// Blocks of the router: one of up to 32 warps per SM for many tokens, of four
// tokens (a warp each) for few.
constexpr int kMostBlocks = 152;
int tokens_per_block(int T) {
  const int per = (int)(((int64_t)T + kMostBlocks - 1) / kMostBlocks);
  return per < 4 ? 4 : per;
}

template <typename X, int C>
cudaError_t run_score(const ScoreArgs& a, int blocks, int threads, cudaStream_t s) {
  return a.groups > 1 ? launch_overlapped(score_route_kernel<X, C, true>, blocks, threads, 0, s, a)
                      : launch_overlapped(score_route_kernel<X, C, false>, blocks, threads, 0, s, a);
}
template <typename X>
cudaError_t run_score(const ScoreArgs& a, int blocks, int threads, cudaStream_t s) {
  if (a.E <= 32) return run_score<X, 1>(a, blocks, threads, s);
  if (a.E <= 64) return run_score<X, 2>(a, blocks, threads, s);
  if (a.E <= 128) return run_score<X, 4>(a, blocks, threads, s);
  if (a.E <= 256) return run_score<X, 8>(a, blocks, threads, s);
  if (a.E <= 512) return run_score<X, 16>(a, blocks, threads, s);
  return run_score<X, 32>(a, blocks, threads, s);
}

}  // namespace

size_t router_workspace_bytes(const moe_router_dims& d) {
  const int per = tokens_per_block(d.T);
  const size_t nb = ((size_t)d.T + per - 1) / per;
  return 16 + nb * d.E * sizeof(int32_t);
}

cudaError_t launch_router(const moe_router_dims& d, const void* logits, const float* bias, const moe_route_out& o,
                          int32_t* hist, int32_t* status, cudaStream_t s) {
  const int per = tokens_per_block(d.T);
  const int nb = (int)(((int64_t)d.T + per - 1) / per);
  const int64_t max_rows = (int64_t)d.T * d.top_k + (int64_t)kAlign * d.E;
  if (nb > 0) {
    const ScoreArgs a{logits, bias, d.ld, d.T, d.E, d.top_k, per, d.groups, d.E / d.groups, d.top_groups,
                      d.group_top, d.score == MOE_SCORE_SIGMOID, d.renormalise != 0, d.scale, o.topk_idx, o.gate,
                      hist, status};
    const int threads = 32 * (per < 32 ? per : 32);
    const cudaError_t e = d.type == MOE_TYPE_BF16 ? run_score<__nv_bfloat16>(a, nb, threads, s)
                                                  : run_score<float>(a, nb, threads, s);
    if (e != cudaSuccess) return e;
  }
  const PlaceArgs p{o.topk_idx, hist, d.T * d.top_k, d.E, nb, per * d.top_k, max_rows, o.counts, o.offsets,
                    o.padded_offsets, o.row_of_assign, o.assign_of_row, status};
  const int64_t fill = ((int64_t)kAlign * d.E + 8191) / 8192;
  static CtxCache<int> cache;
  int set;
  const cudaError_t e = cache.get(&set, [](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32 * kMaxE * 2);
  });
  if (e != cudaSuccess) return e;
  return launch_overlapped(place_kernel, nb + (unsigned)fill, 1024, 32 * d.E * sizeof(uint16_t), s, p);
}

cudaError_t launch_router_backward(const moe_router_dims& d, const moe_route_out& o, const void* logits,
                                   const float* dgate, void* dlogits, int32_t* status, cudaStream_t s) {
  if (d.T == 0) return cudaSuccess;
  const ScoreBwdArgs a{logits, o.topk_idx, o.gate, dgate, dlogits, d.ld, d.T, d.E, d.top_k,
                       d.score == MOE_SCORE_SIGMOID, d.renormalise != 0, d.scale, status};
  const int blocks = (d.T - 1) / 8 + 1, most = kMostBlocks * 8;
  const int grid = blocks < most ? blocks : most;
  return d.type == MOE_TYPE_BF16
             ? launch_overlapped(score_route_backward_kernel<__nv_bfloat16>, grid, 256, 0, s, a)
             : launch_overlapped(score_route_backward_kernel<float>, grid, 256, 0, s, a);
}

cudaError_t launch_balance_bias(const int32_t* counts, int E, float rate, const float* bias, float* out,
                                cudaStream_t s) {
  return launch_overlapped(balance_bias_kernel, 1, 256, 0, s, counts, E, rate, bias, out);
}

}  // namespace moe
