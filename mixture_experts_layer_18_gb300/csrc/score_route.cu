// score_route.cu - routing by scores: softmax or sigmoid scores, a bias for
// balance, groups of experts, top-k, gates; its backward; the bias' update.
//
//   s = softmax(l) or 1 / (1 + exp(-l)),  u = s + bias
//   a group's value is the sum of its `group_top` largest u; the `top_groups`
//   best groups stay; the k largest u in them are chosen (ties: the lower
//   index), and gate_j = scale s_j, or scale s_j / sum of the chosen s.
//
// The choice is that of u in 64 bits, whatever the GPU, found in steps:
//   - keys of 32 bits that hold the leading bits of u in fp32 and the expert's
//     index, so that a round of the choice is one maximum over the lanes (comparing
//     values and indices took 750 instructions a token of 128 experts; 290 with keys, 240
//     where lanes sort theirs, score_many.cu);
//   - where these bits and the error of fp32 (near_of, near_pair) leave it open, the
//     candidates in full fp32, and those that are still too close in pairs of fp32
//     numbers (order; a few tokens in a thousand with 256 sigmoid scores, one in a
//     thousand in pairs);
//   - more candidates than fit: the row's values again with all bits (choose32);
//   - what pairs do not tell (equal sums of different parts): the row in 64 bits
//     (choose64).  This GPU's fp64 takes 43 us for a row of 256.
// Without a bias u orders as the logits do, which are compared themselves.
//
// One warp per token, C neighbouring experts per lane, so that a group is a
// segment of lanes and the logits arrive in vectors; for many tokens eight lanes
// per token (score_many.cu).  Then a second launch gives the assignments their rows
// (for at most kFusedTokens the same one does).
//
// Measured (GB300, fp32 logits, top 8, with the permutation): 1 token of 256 experts
// in 8 groups 5.5 us; 1500 tokens 15 us; 16384 tokens 23 us; 65536 tokens of 128 experts,
// softmax with a bias, 36 us (logits from HBM: 5 us).  The choice is bound by
// instructions with 65536 tokens (59% of the issue slots); with 16384 of 256 experts by the
// latency of what a warp does in turn and by its split (35%: a block has 27 units of four
// tokens for 16 warps, which is what the registers leave room for, so some warps take two);
// the permutation (6 us) by its chain of dependent steps, 4000 cycles of it the other
// blocks' histograms.  What does not fit eight lanes per token, 16384 tokens: 384 experts,
// sigmoid with a bias, 52 us; 512, top 10, softmax, 39; 1024 96; 256, top 16, 44.
//
// Values that fp32 cannot order cost more.  A third of 16384 tokens with logits of zero: 134
// us instead of 23 in 8 groups of 256 experts, 36 instead of 15 without a bias (128
// experts; both look at such a token by a whole warp, choose32), no difference without
// groups and with a bias.
#include "score_route.cuh"

namespace moe {

namespace {

// Rows of the tokens [t0, t1) of one block: run[e] is the row of expert e's next
// assignment.  A token chooses an expert at most once, so the rank of an
// assignment is the number of earlier tokens with the same expert: a bit per token
// and expert, set in any order, counted up to the token's own.
struct PlaceArgs {
  const int32_t* idx;
  const uint16_t* hist;      // [nb][padded4(E)]
  int T, k, E, nb, per_block, words;
  int64_t max_rows, sure;    // rows at or past `sure` belong to no expert, whatever the routing
  int32_t* counts;
  int32_t* offsets;
  int32_t* padded;
  int32_t* row_of;
  int32_t* assign_of;
  unsigned long long inv_k;  // 2^32 / k, rounded up: i inv_k >> 32 is i / k for i k < 2^32
};

constexpr int kPerThread = 8;
__device__ __forceinline__ void place_tokens(const PlaceArgs& a, const int32_t* all_idx, int64_t t0, int64_t t1, int* run,
                                             uint32_t* bits) {
  const int round = 32 * a.words;
  int* first = reinterpret_cast<int*>(bits) + a.words * a.E;   // [words][E]: the row of a word's first assignment
  for (int64_t base = t0; base < t1; base += round) {
    const int n = (int)min((int64_t)round, t1 - base), words = (n + 31) >> 5;
    const int32_t* idx = all_idx + base * a.k;
    const int m = n * a.k;                                     // (at most kPerThread per thread)
    int e[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      e[j] = -1;
      if (i < m) e[j] = idx[i];
    }
    for (int i = threadIdx.x; i < words * a.E; i += blockDim.x) bits[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (j * (int)blockDim.x >= m) break;
      const int t = (int)((threadIdx.x + j * blockDim.x) * a.inv_k >> 32);
      if (e[j] >= 0) atomicOr(&bits[(t >> 5) * a.E + e[j]], 1u << (t & 31));
    }
    __syncthreads();
    for (int x = threadIdx.x; x < a.E; x += blockDim.x) {
      int row = run[x];
#pragma unroll 4
      for (int w = 0; w < words; ++w) {
        first[w * a.E + x] = row;
        row += __popc(bits[w * a.E + x]);
      }
      run[x] = row;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (j * (int)blockDim.x >= m) break;
      if (e[j] < 0) continue;
      const int i = threadIdx.x + j * blockDim.x, t = (int)(i * a.inv_k >> 32), at = (t >> 5) * a.E + e[j];
      const int row = first[at] + __popc(bits[at] & ((1u << (t & 31)) - 1u));
      a.row_of[base * a.k + i] = row;
      a.assign_of[row] = (int)(base * a.k + i);
    }
    if (base + round < t1) __syncthreads();                    // (bits are written again)
  }
}

// Exclusive sums over the experts of their counts (off, where `both`) and of these
// rounded up to kAlign (start): [E + 1] in shared memory, by the whole block (sm: 32).
__device__ __forceinline__ void scan_experts(const int* cnt, int E, bool both, int* off, int* start, int2* sm) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int2 before = make_int2(0, 0);
  for (int c0 = 0; c0 < E; c0 += blockDim.x) {
    const int used = (min(E - c0, (int)blockDim.x) + 31) >> 5;        // warps with experts
    const int e = c0 + threadIdx.x, n = e < E ? cnt[e] : 0, p = (n + kAlign - 1) / kAlign * kAlign;
    int x = n, y = p;
    if (w < used) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, y, o);
        if (lane >= o) y += v;
      }
      if (both) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(kAll, x, o);
          if (lane >= o) x += u;
        }
      }
      if (lane == 31) sm[w] = make_int2(x, y);
    }
    __syncthreads();
    if (w < used) {
      int2 all = lane < used ? sm[lane] : make_int2(0, 0), mine = lane < w ? all : make_int2(0, 0);
      all.y = __reduce_add_sync(kAll, all.y);
      mine.y = __reduce_add_sync(kAll, mine.y);
      if (e < E) start[e] = before.y + mine.y + y - p;
      if (both) {
        all.x = __reduce_add_sync(kAll, all.x);
        mine.x = __reduce_add_sync(kAll, mine.x);
        if (e < E) off[e] = before.x + mine.x + x - n;
      }
      before.x += all.x;
      before.y += all.y;
    }
    if (c0 + (int)blockDim.x < E) __syncthreads();    // (sm is written again; all warps are used but in the last part)
  }
  if (threadIdx.x == 0) {
    off[E] = before.x;
    start[E] = before.y;
  }
  __syncthreads();
}

// assign_of_row = -1 in [r0, r1), by blocks `b` of `nb`.
__device__ __forceinline__ void no_assignment(const PlaceArgs& a, int64_t r0, int64_t r1, int b, int nb) {
  const int64_t v0 = (r0 + 3) / 4 * 4;
  if (b == 0 && threadIdx.x < 4 && r0 + threadIdx.x < min(v0, r1)) a.assign_of[r0 + threadIdx.x] = -1;
  for (int64_t r = v0 + ((int64_t)b * blockDim.x + threadIdx.x) * 4; r < r1; r += (int64_t)nb * blockDim.x * 4) {
    if (r + 4 <= r1) {
      *reinterpret_cast<int4*>(a.assign_of + r) = make_int4(-1, -1, -1, -1);
    } else {
      for (int64_t i = r; i < r1; ++i) a.assign_of[i] = -1;
    }
  }
}

// Rows without an assignment: those behind each expert's (a warp per expert), and behind the last.
__device__ __forceinline__ void fill_rows(const PlaceArgs& a, const int* cnt, const int* start, int b, int nb) {
  const int w = threadIdx.x >> 5, nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  for (int e = b * nw + w; e < a.E; e += nb * nw)
    for (int r = start[e] + cnt[e] + lane; r < start[e + 1]; r += 32) a.assign_of[r] = -1;
  no_assignment(a, start[a.E], a.max_rows, b, nb);
}

// Threads of a block at most: the keys of wider rows take more registers.
template <int C>
constexpr int kRouteThreads = C <= 4 ? 1024 : C <= 8 ? 768 : C <= 16 ? 512 : 256;

// With p.nb 1 the first block has all tokens (few of them) and places them too,
// without a second launch; the others fill the rows from p.sure on, which no routing reaches.
template <typename X, int C, bool GROUPED>
__global__ void __launch_bounds__(kRouteThreads<C>) score_route_kernel(const __grid_constant__ ScoreArgs a,
                                                           const __grid_constant__ PlaceArgs p) {
  __shared__ int hist[kMaxE];
  __shared__ uint2 slots[32][33];
  __shared__ int2 scan[32];
  extern __shared__ uint32_t dyn[];
  int* chosen = reinterpret_cast<int*>(dyn) + (3 + 2 * p.words) * a.E + 2;    // [T][k], with p.nb 1
  let_next_start();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  wait_for_previous();
  if (p.nb == 1 && blockIdx.x > 0) {
    no_assignment(p, p.sure, p.max_rows, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  uint2* slot = slots[threadIdx.x >> 5];
  const int64_t t0 = (int64_t)blockIdx.x * a.per_block;
  const int64_t t1 = min((int64_t)a.T, t0 + a.per_block);
  const bool by_logit = !a.bias && (!GROUPED || a.group_top == 1);
  constexpr uint32_t kIndex = 32 * C - 1;               // the bits of a key that hold the index
  constexpr float kLead = 32.f * C * 0x1p-23f;          // what they take from the value, relative to it
  constexpr bool kLossless = sizeof(X) == 2;            // a bf16 logit is all leading bits
  auto leading = [](uint32_t key) {
    const uint32_t k = key & ~kIndex;
    return k > 0x007fffffu ? value_of(k) : -INFINITY;   // (-inf, and none)
  };
  int64_t t = t0 + (threadIdx.x >> 5);
  Logits<X, C> next;
  if (t < t1) next.load(static_cast<const X*>(a.logits) + t * a.ld, a.E, a.vec);
  float bias[C], bias_most = 0.f;
  bool bad = false, unused = false;
#pragma unroll
  for (int q = 0; q < C; ++q) bias[q] = 0.f;
  if (a.bias && t < t1) {
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int e = lane * C + q;
      const float b = e < a.E ? a.bias[e] : 0.f;
      if (fabsf(b) < INFINITY) bias[q] = b;
      else bad = true;
      bias_most = fmaxf(bias_most, fabsf(bias[q]));
    }
    bias_most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(bias_most)));
  }
  for (; t < t1; t += nw) {
    const X* row = static_cast<const X*>(a.logits) + t * a.ld;
    const Logits<X, C> raw = next;
    if (t + nw < t1) next.load(row + nw * a.ld, a.E, a.vec);
    float u[C], finite = 0.f;
#pragma unroll
    for (int q = 0; q < C; ++q) {
      u[q] = lane * C + q < a.E ? raw.get(q) : 0.f;
      finite = fmaf(u[q], 0.f, finite);               // NaN after an infinity or a NaN
    }
    const bool plain = !__any_sync(kAll, finite != 0.f);   // (E < 32 C: with zeros behind the last)
    if (!plain || a.E < 32 * C) {
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const bool there = lane * C + q < a.E;
        if (there && !(u[q] < INFINITY)) bad = true;       // NaN and +inf read as -inf
        if (!there || !(u[q] < INFINITY)) u[q] = -INFINITY;
      }
    }
    float top = 0.f, sum = 1.f;
    if (!a.sigmoid && (!by_logit || !a.renorm)) softmax_of(u, &top, &sum);
    const float inv = a.sigmoid ? 1.f : __fdividef(1.f, sum);
    // the keys: leading bits of the value, then the index, downwards
    uint32_t key[C], f1 = 0, f2 = 0;         // (f1, f2: the lane's best two values, all bits)
#pragma unroll
    for (int q = 0; q < C; ++q) {
      float v = u[q];
      if (!by_logit) {
        v = score_of(a, v, top, inv) + bias[q];
        if (!plain && !(u[q] > -INFINITY)) v = -INFINITY;
      }
      uint32_t k = key_of(v);
      if (a.E < 32 * C && lane * C + q >= a.E) k = 0;
      if (GROUPED) {
        f2 = max(f2, min(f1, k));
        f1 = max(f1, k);
      }
      key[q] = k ? (k & ~kIndex) | (kIndex - q - lane * C) : 0;
    }
    bool again = false;
    uint32_t m1 = 0, m2 = 0;                 // the lane's best two keys
    auto best_two = [&]() {
      m1 = key[0];
      m2 = 0;
#pragma unroll
      for (int q = 1; q < C; ++q) {
        m2 = max(m2, min(m1, key[q]));
        m1 = max(m1, key[q]);
      }
    };
    if (!GROUPED || a.seg) best_two();
    if (GROUPED) {
      float mine = -INFINITY;              // lanes of group g (seg > 0) or lane g: its value
      uint32_t g1 = f1, g2 = f2;
      if (a.seg) {                         // a group is a whole number of lanes, a power of two
        for (int o = 1; o < a.seg; o <<= 1) {
          const uint32_t n1 = __shfl_xor_sync(kAll, g1, o), n2 = __shfl_xor_sync(kAll, g2, o);
          g2 = max(min(g1, n1), max(g2, n2));
          g1 = max(g1, n1);
        }
        if (lane < a.groups << a.seg_log) mine = a.group_top == 1 ? value_of(g1) : value_of(g1) + value_of(g2);
      } else {
        for (int g = 0; g < a.groups; ++g) {
          uint32_t b1 = 0, b2 = 0;
#pragma unroll
          for (int q = 0; q < C; ++q) {
            const int e = lane * C + q;
            if (e >= g * a.group_size && e < (g + 1) * a.group_size) {
              b2 = max(b2, min(b1, key[q]));
              b1 = max(b1, key[q]);
            }
          }
          const uint32_t f = __reduce_max_sync(kAll, b1);
          float v = leading(f);
          if (a.group_top > 1) v += leading(__reduce_max_sync(kAll, b1 == f ? b2 : b1));
          if (lane == g) mine = v;
        }
      }
      const int own = a.seg ? lane >> a.seg_log : lane;
      int better = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float v = __shfl_sync(kAll, mine, a.seg ? g << a.seg_log : g);
        better += v > mine || (v == mine && g < own);
      }
      bool stays = own < a.groups && better < a.top_groups;
      if (a.top_groups < a.groups) {
        const float lo = -value_of(__reduce_max_sync(kAll, stays ? key_of(-mine) : 0x007fffffu));   // (-inf)
        const float hi = value_of(__reduce_max_sync(kAll, own < a.groups && !stays ? key_of(mine) : 0x007fffffu));
        // (from leading bits a value is up to kLead of itself lower)
        const float most = bias_most + (a.sigmoid ? 1.f : inv);
        const float gap = by_logit ? 0.f : 2.f * near_of<C>(a.sigmoid, inv, 2.f * most) + (a.seg ? 0.f : 2.f * kLead * most);
        again = hi > -INFINITY && !(lo - hi > gap || (by_logit && (kLossless || a.seg)));
        if (again && a.seg && !by_logit) {
          // the group's best by their keys, if no third one comes near the last of them
          uint32_t b1 = m1, b2 = m2;
          for (int o = 1; o < a.seg; o <<= 1) {
            const uint32_t n1 = __shfl_xor_sync(kAll, b1, o), n2 = __shfl_xor_sync(kAll, b2, o);
            b2 = max(min(b1, n1), max(b2, n2));
            b1 = max(b1, n1);
          }
          const float last = leading(a.group_top == 1 ? b1 : b2);
          const float floor = last - near_of<C>(a.sigmoid, inv, last) - kLead * fabsf(last);
          int count = 0;
#pragma unroll
          for (int q = 0; q < C; ++q) count += leading(key[q]) >= floor;
          for (int o = 1; o < a.seg; o <<= 1) count += __shfl_xor_sync(kAll, count, o);
          const bool live = own < a.groups && last > -INFINITY;
          const int e0 = kIndex - (b1 & kIndex), e1 = kIndex - (b2 & kIndex);
          bool unsure = live && count > a.group_top;
          stays = better_groups(a, live ? logit(a, row, e0, &bad) : 0.f, live ? bias_of(a, e0) : 0.f,
                                live && b2 ? logit(a, row, e1, &bad) : 0.f, live && b2 ? bias_of(a, e1) : 0.f, live, own, 0,
                                a.seg_log, top, a.sigmoid ? Pair{} : softmax_scale(a, row, top), &unsure);
          again = __any_sync(kAll, unsure);
        }
      }
      if (a.seg) {
        if (!stays) m1 = m2 = 0;
      } else {
        const unsigned stay = __ballot_sync(kAll, stays);
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const int e = lane * C + q;
          if (e < a.E && !(stay >> (e / a.group_size) & 1u)) key[q] = 0;
        }
        best_two();
      }
    }
    // rounds of a warp maximum: k, and more while the next may be as good as the k-th
    uint32_t sel = 0;
    float last = -INFINITY;
    int n = 0;
    for (; n < 32; ++n) {
      const uint32_t m = __reduce_max_sync(kAll, m1);
      if (n >= a.k) {
        const float v = leading(m);
        const float gap = by_logit ? 0.f : near_of<C>(a.sigmoid, inv, fmaxf(fabsf(last), fabsf(v))) + kLead * fabsf(v);
        if ((by_logit && kLossless) || !(v > -INFINITY) || last - v > gap) break;
      } else if (n == a.k - 1) {
        last = leading(m);
      }
      if (lane == n) sel = m;
      if (m1 == m) {
        m1 = m2;
        m2 = 0;
        if (m1 == 0) {                       // the third, and so on
#pragma unroll
          for (int q = 0; q < C; ++q)
            if (key[q] < m) m1 = max(m1, key[q]);
        }
      }
    }
    int sel_e = sel ? kIndex - (sel & kIndex) : 0;
    float l = -INFINITY;
    if (sel) l = logit(a, row, sel_e, &unused);
    if (!(by_logit && kLossless)) {
      // is the order of neighbours certain?  (Equal ones are in it.)
      const float v = leading(sel), pv = __shfl_up_sync(kAll, v, 1), pl = __shfl_up_sync(kAll, l, 1);
      float b = 0.f;
      if (a.bias && sel) b = bias_of(a, sel_e);
      const float pb = __shfl_up_sync(kAll, b, 1);
      const float gap = by_logit ? 0.f : near_pair<C>(a.sigmoid, inv, pv, pb, v, b) + 2.f * kLead * fabsf(v);
      const bool close = lane > 0 && v > -INFINITY && !(pv - v > gap) && !(pl == l && pb == b);
      if (again || n == 32) {
        sel_e = choose32<X, C, GROUPED>(a, row, slot);
        if (lane < a.k) l = logit(a, row, sel_e, &unused);
      } else if (__any_sync(kAll, close) || n > a.k) {
        const int e = order<X, C>(a, row, sel_e, l, b, n, top, inv, slot);
        sel_e = __any_sync(kAll, e < 0) ? choose64<X, C>(a, row) : e;
        if (lane < a.k) l = logit(a, row, sel_e, &unused);
      }
    }
    if (lane >= a.k) l = -INFINITY;
    // gates
    const bool none = !__any_sync(kAll, l > -INFINITY);
    float w = !(l > -INFINITY) ? 0.f : a.sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - top);
    if (a.renorm) {
      // relative to the largest chosen score for the softmax, and where a sigmoid leaves the range of
      // fp32's normal numbers (below e^-87), which its gate need not do
      if (!a.sigmoid || __any_sync(kAll, l > -INFINITY && l < -87.f)) {
        const float x = a.sigmoid ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;      // log s (+ a constant)
        const float m = value_of(__reduce_max_sync(kAll, key_of(x)));
        w = l > -INFINITY ? expf(x - m) : 0.f;
      }
      float all = w;
      if (a.k > 8) {
        all += __shfl_xor_sync(kAll, all, 16);
        all += __shfl_xor_sync(kAll, all, 8);
      }
#pragma unroll
      for (int o = 4; o; o >>= 1) all += __shfl_xor_sync(kAll, all, o);
      w = w / all;
    } else if (!a.sigmoid) {
      w = w / sum;
    }
    if (none) bad = true;
    if (lane < a.k) {
      a.idx[t * a.k + lane] = sel_e;
      if (p.nb == 1) chosen[t * a.k + lane] = sel_e;
      a.gate[t * a.k + lane] = none ? 0.f : a.scale * w;
      atomicAdd(&hist[sel_e], 1);
    }
  }
  if (bad) report(a.status, MOE_ERR_BAD_INPUT);
  __syncthreads();
  if (p.nb == 1) {
    int* off = reinterpret_cast<int*>(dyn);
    int* start = off + a.E + 1;
    int* run = start + a.E + 1;
    scan_experts(hist, a.E, true, off, start, scan);
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
      if (e < a.E) {
        run[e] = start[e];
        p.counts[e] = hist[e];
      }
      p.offsets[e] = off[e];
      p.padded[e] = start[e];
    }
    // (no row has its assignment before place_tokens' barriers)
    no_assignment(p, 0, gridDim.x > 1 ? p.sure : p.max_rows, 0, 1);
    __syncthreads();
    place_tokens(p, chosen, 0, a.T, run, reinterpret_cast<uint32_t*>(run + a.E));
  } else {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * padded4(a.E) + e] = (uint16_t)hist[e];
  }
}

// ---------------------------------------------------------- permutation
// Blocks [0, nb): rows of this block's assignments.  Every block adds the
// router's histograms up by itself (their sum over all blocks gives the rows'
// start of each expert, that over the blocks before it its own share), which
// saves a launch between the two.  Blocks from nb on: the rows without an assignment.
constexpr int kPlaceThreads = 512;
__global__ void __launch_bounds__(kPlaceThreads) place_kernel(const __grid_constant__ PlaceArgs a) {
  __shared__ int cnt[kMaxE], run[kMaxE], off[kMaxE + 1], start[kMaxE + 1];
  __shared__ int2 scan[32];
  extern __shared__ uint32_t dyn[];
  let_next_start();
  const int b = blockIdx.x;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = run[e] = 0;
  __syncthreads();
  wait_for_previous();
  // threads (slice, four experts): each adds up some of the histograms, all loads at once
  const int four = padded4(a.E) / 4, slices = (int)blockDim.x / four, slice = threadIdx.x / four;
  const int e4 = threadIdx.x % four * 4;
  if (slice < slices) {
    int4 total = make_int4(0, 0, 0, 0), before = total;
    const uint2* h = reinterpret_cast<const uint2*>(a.hist) + threadIdx.x % four;
    for (int i0 = slice; i0 < a.nb; i0 += 10 * slices) {       // ten loads at once, whatever is left
      uint2 c[10];
#pragma unroll
      for (int j = 0; j < 10; ++j) {
        const int i = i0 + j * slices;
        c[j] = i < a.nb ? h[(int64_t)i * four] : make_uint2(0, 0);
      }
#pragma unroll
      for (int j = 0; j < 10; ++j) {
        const int4 d = make_int4(c[j].x & 0xffff, c[j].x >> 16, c[j].y & 0xffff, c[j].y >> 16);
        total.x += d.x; total.y += d.y; total.z += d.z; total.w += d.w;
        if (i0 + j * slices < b) {
          before.x += d.x; before.y += d.y; before.z += d.z; before.w += d.w;
        }
      }
    }
    // (elements behind E are not written: they belong to no expert)
    const int t[4] = {total.x, total.y, total.z, total.w}, f[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e4 + i < a.E) {
        atomicAdd(&cnt[e4 + i], t[i]);
        if (b < a.nb) atomicAdd(&run[e4 + i], f[i]);
      }
  }
  __syncthreads();
  scan_experts(cnt, a.E, b == 0, off, start, scan);
  if (b == 0)
    for (int i = threadIdx.x; i <= a.E; i += blockDim.x) {
      if (i < a.E) a.counts[i] = cnt[i];
      a.offsets[i] = off[i];
      a.padded[i] = start[i];
    }
  if (b >= a.nb) {
    fill_rows(a, cnt, start, b - a.nb, gridDim.x - a.nb);
    return;
  }
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) run[i] += start[i];
  __syncthreads();
  const int64_t t0 = (int64_t)b * a.per_block;
  place_tokens(a, a.idx, t0, min((int64_t)a.T, t0 + a.per_block), run, dyn);
}

// -------------------------------------------------------------- backward
struct ScoreBwdArgs {
  const void* logits;
  const int32_t* idx;
  const float* gate;
  const float* dgate;
  void* dlogits;
  int64_t ld;
  int T, E, k, sigmoid, renorm, vec;
  float inv_scale;
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
      // (rounded product by product: of one expert alone this is what rounding leaves of 0)
      d = a.renorm ? w * __fsub_rn(dw, __fmul_rn(inner, a.inv_scale)) : w * dw;
      if (a.sigmoid && e >= 0) {
        const float v = to_f(row[e]);
        d *= v < INFINITY ? 1.f / (1.f + expf(v)) : 1.f;                     // 1 - s
      }
      if (a.vec) {
        for (int c = lane; c < a.E * (int)sizeof(X) / 16; c += 32) reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
      } else {
        for (int c = lane; c < a.E; c += 32) put(out + c, 0.f);
      }
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
// tokens (a warp each) for few; one block that places its tokens too for at most
// kFusedTokens.  (More than 65535 would not fit the histograms' 16 bits.)  kMostBlocks is
// this GPU's number of SMs: where fewer are at hand the last blocks run after the others, with
// the same results; the workspace has room for that many on any device.
constexpr int kMostBlocks = 152, kFusedTokens = 32;
int tokens_per_block(int T) {
  const int per = (int)(((int64_t)T + kMostBlocks - 1) / kMostBlocks);
  return T <= kFusedTokens ? kFusedTokens : per < 4 ? 4 : per > 65535 ? 65535 : per;
}

// Words of 32 tokens that a round of the placement takes by blocks of `threads`:
// what a block has, up to 28 KB of bits and rows, and kPerThread assignments per thread.
int place_words(int per_block, int E, int k, int threads) {
  int n = (per_block + 31) / 32;
  if (n > 3584 / E) n = 3584 / E;
  if (n > threads * kPerThread / (32 * k)) n = threads * kPerThread / (32 * k);
  return n;
}

template <typename X, int C, bool GROUPED>
cudaError_t run_score(ScoreArgs a, const PlaceArgs& p, int blocks, cudaStream_t s) {
  constexpr int kVec = C * (int)sizeof(X) < 16 ? C * (int)sizeof(X) : 16;
  a.vec = kVec >= 4 && ((uintptr_t)a.logits & (kVec - 1)) == 0 && a.ld * sizeof(X) % kVec == 0 &&
          a.E * sizeof(X) % kVec == 0;
  a.seg = a.group_size % C ? 0 : a.group_size / C;
  if (a.seg & (a.seg - 1)) a.seg = 0;
  for (a.seg_log = 0; 1 << a.seg_log < a.seg;) ++a.seg_log;
  const int warps = blocks == 1 ? a.T : a.per_block, most = kRouteThreads<C>;
  if (blocks == 1) {
    const int threads = warps < 8 ? 256 : 32 * warps > most ? most : 32 * warps;
    const int smem = ((3 + 2 * p.words) * a.E + 2 + a.T * a.k) * 4;
    return launch_overlapped(score_route_kernel<X, C, GROUPED>, 1 + (unsigned)((p.max_rows - p.sure) / 4096),
                             threads, smem, s, a, p);
  }
  const int threads = 32 * warps > most ? most : 32 * warps;
  return launch_overlapped(score_route_kernel<X, C, GROUPED>, blocks, threads, 0, s, a, p);
}
template <typename X, int C>
cudaError_t run_score(const ScoreArgs& a, const PlaceArgs& p, int blocks, cudaStream_t s) {
  return a.groups > 1 ? run_score<X, C, true>(a, p, blocks, s) : run_score<X, C, false>(a, p, blocks, s);
}
template <typename X>
cudaError_t run_score(const ScoreArgs& a, const PlaceArgs& p, int blocks, cudaStream_t s) {
  bool taken;
  const cudaError_t e = launch_score_many<X>(a, blocks, &taken, s);
  if (e != cudaSuccess || taken) return e;
  if (a.E <= 32) return run_score<X, 1>(a, p, blocks, s);
  if (a.E <= 64) return run_score<X, 2>(a, p, blocks, s);
  if (a.E <= 128) return run_score<X, 4>(a, p, blocks, s);
  if (a.E <= 256) return run_score<X, 8>(a, p, blocks, s);
  if (a.E <= 512) return run_score<X, 16>(a, p, blocks, s);
  return run_score<X, 32>(a, p, blocks, s);
}

}  // namespace

size_t router_workspace_bytes(const moe_router_dims& d) {
  const int per = tokens_per_block(d.T);
  const size_t nb = ((size_t)d.T + per - 1) / per;
  return 16 + nb * padded4(d.E) * sizeof(uint16_t);
}

cudaError_t launch_router(const moe_router_dims& d, const void* logits, const float* bias, const moe_route_out& o,
                          uint16_t* hist, int32_t* status, cudaStream_t s) {
  const int per = tokens_per_block(d.T);
  const int nb = (int)(((int64_t)d.T + per - 1) / per);
  const int64_t max_rows = (int64_t)d.T * d.top_k + (int64_t)kAlign * d.E;
  const int words = place_words(per, d.E, d.top_k, nb == 1 ? 256 : kPlaceThreads);
  const int64_t n = (int64_t)d.T * d.top_k, sure = n + (kAlign - 1) * (n < d.E ? n : d.E);
  const PlaceArgs p{o.topk_idx, hist, d.T, d.top_k, d.E, nb, per, words, max_rows, sure, o.counts, o.offsets,
                    o.padded_offsets, o.row_of_assign, o.assign_of_row, ((1ull << 32) + d.top_k - 1) / d.top_k};
  if (nb > 0) {
    const ScoreArgs a{logits, bias, d.ld, d.T, d.E, d.top_k, per, d.groups, d.E / d.groups, d.top_groups,
                      d.group_top, 0, 0, d.score == MOE_SCORE_SIGMOID, d.renormalise != 0, 0, d.scale, o.topk_idx,
                      o.gate, hist, status};
    const cudaError_t e = d.type == MOE_TYPE_BF16 ? run_score<__nv_bfloat16>(a, p, nb, s) : run_score<float>(a, p, nb, s);
    if (e != cudaSuccess || nb == 1) return e;
  }
  const int fill = (d.E + kPlaceThreads / 32 - 1) / (kPlaceThreads / 32);      // (a warp per expert)
  return launch_overlapped(place_kernel, (unsigned)(nb + fill), kPlaceThreads, 2 * words * d.E * 4, s, p);
}

cudaError_t launch_router_backward(const moe_router_dims& d, const moe_route_out& o, const void* logits,
                                   const float* dgate, void* dlogits, int32_t* status, cudaStream_t s) {
  if (d.T == 0) return cudaSuccess;
  const int vec = ((uintptr_t)dlogits & 15) == 0 && d.E * (d.type == MOE_TYPE_BF16 ? 2 : 4) % 16 == 0;
  const ScoreBwdArgs a{logits, o.topk_idx, o.gate, dgate, dlogits, d.ld, d.T, d.E, d.top_k,
                       d.score == MOE_SCORE_SIGMOID, d.renormalise != 0, vec, 1.f / d.scale, status};
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
