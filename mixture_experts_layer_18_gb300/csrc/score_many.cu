// score_many.cu - the router by scores (score_route.cu) for many tokens: 23 us for 16384
// tokens of 256 experts in groups and 36 for 65536 of 128, with the permutation, where a
// warp per token took 36 and 69.
#include "score_route.cuh"

namespace moe {

namespace {

// Many tokens: eight lanes per token, four tokens per warp, so that what a token
// takes besides its elements (order, gates, addresses) is paid once for four.
// A group has a power of two of the eight lanes (all of them without groups), and a
// lane up to CL neighbouring experts of its group; top_k <= 8.  A lane puts its keys
// in order by eights and keeps the best eight, and the lanes' lists are merged in three
// steps: 10 % less time than a maximum over the lanes for each of the chosen, whose
// rounds wait for one another (65536 tokens of 128 experts: 36.1 us instead of 39.1).
__device__ __forceinline__ uint32_t max8(uint32_t v) {          // over a token's lanes
#pragma unroll
  for (int o = 4; o; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// softmax_scale of the tokens with a lane in `open`, a token at a time by the whole warp.
template <typename X>
__device__ __forceinline__ Pair softmax_scales(const ScoreArgs& a, const X* row, float top, unsigned open) {
  Pair scale{};
  for (int t = 0; t < 32; t += 8)
    if (open >> t & 0xffu) {
      const X* r = reinterpret_cast<const X*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(row), t));
      const Pair p = softmax_scale(a, r, __shfl_sync(kAll, top, t));
      if ((threadIdx.x & 24) == t) scale = p;
    }
  return scale;
}

// As order(), for up to 16 candidates of each of four tokens: lane sl of a token
// has candidates sl and sl + 8 (n: how many the token has).  Returns the lane's
// expert in that order, -1 to all lanes of a token whose order is not known.
template <typename X, int CL>
__device__ __noinline__ int order8(const ScoreArgs& a, const X* row, int e0, int e1, float l0, float l1, float b0, float b1,
                                   int n, float top, float inv, int* slot) {
  const int e[2] = {e0, e1};
  const float l[2] = {l0, l1}, b[2] = {b0, b1};
  const int sl = threadIdx.x & 7, first = threadIdx.x & 24;
  const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
  float v[2];
  bool on[2];
  int better[2] = {0, 0};
  bool unsure = false;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    on[r] = sl + 8 * r < n && l[r] > -INFINITY;
    v[r] = !on[r] || by_logit ? l[r] : score_of(a, l[r], top, inv) + b[r];
  }
  const int most = (int)__reduce_max_sync(kAll, (unsigned)n);
  for (int i = 0; i < most; ++i) {
    const int at = first + (i & 7);
    const float ov = __shfl_sync(kAll, i < 8 ? v[0] : v[1], at), ol = __shfl_sync(kAll, i < 8 ? l[0] : l[1], at);
    const float ob = __shfl_sync(kAll, i < 8 ? b[0] : b[1], at);
    const int oe = __shfl_sync(kAll, i < 8 ? e[0] : e[1], at);
    const bool other = ol > -INFINITY;
    if (i >= n) continue;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (sl + 8 * r >= n || oe == e[r]) continue;
      const float gap = near_pair<CL>(a.sigmoid, inv, v[r], b[r], ov, ob);
      if ((ol == l[r] && ob == b[r]) || (!on[r] && !other)) better[r] += oe < e[r];
      else if (!on[r] || !other) better[r] += other;               // masked ones last
      else if (by_logit || fabsf(ov - v[r]) > gap) better[r] += ov > v[r] || (ov == v[r] && oe < e[r]);
      else unsure = true;
    }
  }
  unsigned open = __ballot_sync(kAll, unsure);
  if (open) {
    const Pair scale = a.sigmoid ? Pair{} : softmax_scales(a, row, top, open);
    const Exact x0 = exact_value(a.sigmoid, l[0], b[0], top, scale), x1 = exact_value(a.sigmoid, l[1], b[1], top, scale);
    better[0] = better[1] = 0;
    unsure = false;
    for (int i = 0; i < most; ++i) {
      const int at = first + (i & 7);
      const float oh = __shfl_sync(kAll, i < 8 ? x0.u.h : x1.u.h, at), olow = __shfl_sync(kAll, i < 8 ? x0.u.l : x1.u.l, at);
      const float oo = __shfl_sync(kAll, i < 8 ? x0.off : x1.off, at), ol = __shfl_sync(kAll, i < 8 ? l[0] : l[1], at);
      const float ob = __shfl_sync(kAll, i < 8 ? b[0] : b[1], at), ov = __shfl_sync(kAll, i < 8 ? v[0] : v[1], at);
      const int oe = __shfl_sync(kAll, i < 8 ? e[0] : e[1], at);
      const bool other = ol > -INFINITY;
      if (i >= n) continue;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (sl + 8 * r >= n || oe == e[r]) continue;
        const Exact& x = r ? x1 : x0;
        const float gap = near_pair<CL>(a.sigmoid, inv, v[r], b[r], ov, ob);
        const float d = (oh - x.u.h) + (olow - x.u.l);
        if ((ol == l[r] && ob == b[r]) || (!on[r] && !other)) better[r] += oe < e[r];
        else if (!on[r] || !other) better[r] += other;
        else if (by_logit || fabsf(ov - v[r]) > gap) better[r] += ov > v[r] || (ov == v[r] && oe < e[r]);
        else if (fabsf(d) > oo + x.off) better[r] += d > 0.f;
        else unsure = true;
      }
    }
    open = __ballot_sync(kAll, unsure);
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (sl + 8 * r < n) slot[first * 2 + better[r]] = e[r];
  __syncwarp();
  return open >> first & 0xffu ? -1 : sl < n ? slot[first * 2 + sl] : 0;
}

// Eight keys in descending order: by a merge exchange network (19 exchanges),
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
__device__ __forceinline__ void sort8(uint32_t (&k)[8]) {
  exchange(k[0], k[1]); exchange(k[2], k[3]); exchange(k[4], k[5]); exchange(k[6], k[7]);
  exchange(k[0], k[2]); exchange(k[1], k[3]); exchange(k[4], k[6]); exchange(k[5], k[7]);
  exchange(k[1], k[2]); exchange(k[5], k[6]);
  exchange(k[0], k[4]); exchange(k[1], k[5]); exchange(k[2], k[6]); exchange(k[3], k[7]);
  exchange(k[2], k[4]); exchange(k[3], k[5]);
  exchange(k[1], k[2]); exchange(k[3], k[4]); exchange(k[5], k[6]);
}
// and the best eight of two such lists: one against the other backwards leaves them
// as a list that rises and falls, which three rounds of exchanges put in order.
__device__ __forceinline__ void merge8(uint32_t (&k)[8], const uint32_t (&other)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) k[i] = max(k[i], other[7 - i]);
#pragma unroll
  for (int o = 4; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & o)) exchange(k[i], k[i + o]);
}

// As many warps as the registers leave room for (5000 tokens of 256 experts: 16.8 us
// with 512 threads, 18.0 with 576, 17.1 with 480; 65536 of 128: 36.0 with 736 or 800,
// 36.2 with 640).
template <int CL>
constexpr int kManyThreads = CL > 16 ? 512 : 736;

template <typename X, int CL, bool GROUPED>
__global__ void __launch_bounds__(kManyThreads<CL>, 1) score_many_kernel(const __grid_constant__ ScoreArgs a) {
  constexpr uint32_t kIndex = 8 * CL - 1;               // the bits of a key that hold the expert's place
  constexpr float kLead = 8.f * CL * 0x1p-23f;          // what they take from the value, relative to it
  constexpr bool kLossless = sizeof(X) == 2;            // a bf16 logit is all leading bits
  constexpr int V = CL * (int)sizeof(X) < 16 ? CL : 16 / (int)sizeof(X);
  __shared__ int hist[8 * CL];
  __shared__ float biases[8 * CL];                      // by expert,
  __shared__ __align__(16) float bias[8 * (CL + 4)];    // and by lane (rows apart by 4 banks)
  __shared__ uint2 slots[kManyThreads<CL> / 32][33];
  __shared__ int units;
  let_next_start();
  for (int e = threadIdx.x; e < 8 * CL; e += kManyThreads<CL>) hist[e] = 0;
  if (threadIdx.x == 0) units = 0;
  wait_for_previous();
  bool bad = false, unused = false;
  const bool by_logit = !a.bias && (!GROUPED || a.group_top == 1);
  // the first expert of a lane, and how many it has (the last of a group's lanes may have fewer or none)
  auto first_of = [&](int l) { return (l >> a.seg_log) * a.group_size + (l & (a.seg - 1)) * CL; };
  auto count_of = [&](int l) {
    return l >> a.seg_log < a.groups ? max(0, min(CL, a.group_size - (l & (a.seg - 1)) * CL)) : 0;
  };
  for (int i = threadIdx.x; i < 8 * CL; i += kManyThreads<CL>) {
    const int l = i / CL, q = i % CL, e = first_of(l) + q;
    float b = 0.f;
    if (a.bias && q < count_of(l)) {
      b = bias_of(a, e);
      if (!(fabsf(a.bias[e]) < INFINITY)) bad = true;
    }
    bias[l * (CL + 4) + q] = b;
    if (q < count_of(l)) biases[e] = b;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, sl = lane & 7, first = lane & 24;
  uint2* slot = slots[threadIdx.x >> 5];
  const float* my_bias = bias + sl * (CL + 4);
  const int e0 = first_of(sl), count = count_of(sl);
  const uint32_t index0 = kIndex - sl * CL;             // a key's place of the lane's first expert, downwards
  // the expert of a key (of a masked one, which may be none: some expert)
  auto expert = [&](uint32_t key) {
    const int at = kIndex - (key & kIndex);
    return min(first_of(at / CL) + at % CL, a.E - 1);
  };
  float bias_most = 0.f;
  if (a.bias) {
#pragma unroll
    for (int q = 0; q < CL; ++q) bias_most = fmaxf(bias_most, fabsf(my_bias[q]));
    bias_most = __uint_as_float(max8(__float_as_uint(bias_most)));
  }
  auto leading = [](uint32_t key) {
    const uint32_t k = key & ~kIndex;
    return k > 0x007fffffu ? value_of(k) : -INFINITY;   // (-inf, and none)
  };
  const int64_t t0 = (int64_t)blockIdx.x * a.per_block, t1 = min((int64_t)a.T, t0 + a.per_block);
  for (;;) {
    // warps take the block's tokens as they come: one that has to look closer delays no others
    int unit = 0;
    if (lane == 0) unit = atomicAdd(&units, 1);
    const int64_t tb = t0 + (int64_t)__shfl_sync(kAll, unit, 0) * 4;
    if (tb >= t1) break;
    const int64_t t = min(tb + (lane >> 3), t1 - 1);    // (past the end: the last token again, not stored)
    const bool mine_on = tb + (lane >> 3) < t1;
    const X* row = static_cast<const X*>(a.logits) + t * a.ld;
    float u[CL];
    rows::F2 finite = rows::f2(0.f, 0.f);
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < CL / V; ++i) {
        uint32_t w[4] = {0, 0, 0, 0};
        if (i * V < count) {
          if constexpr (V * sizeof(X) == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + e0 + i * V);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(row + e0 + i * V);
            w[0] = x.x; w[1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
          u[i * V + j] = sizeof(X) == 4 ? __uint_as_float(w[j & 3])
                                        : j & 1 ? bf16_hi(w[(j / 2) & 3]) : bf16_lo(w[(j / 2) & 3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < CL; ++q) u[q] = q < count ? to_f(row[e0 + q]) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < CL; q += 2)                     // NaN after an infinity or a NaN
      finite = rows::fma2(rows::f2(u[q], u[q + 1]), rows::f2(0.f, 0.f), finite);
    const bool plain = !__any_sync(kAll, rows::sum2(finite) != 0.f || count < CL);
    if (!plain) {
#pragma unroll
      for (int q = 0; q < CL; ++q) {
        const bool there = q < count;
        if (there && !(u[q] < INFINITY)) bad = true;    // NaN and +inf read as -inf
        if (!there || !(u[q] < INFINITY)) u[q] = -INFINITY;
      }
    }
    float top = 0.f, sum = 1.f;
    if (!a.sigmoid && (!by_logit || !a.renorm)) {
      float m = u[0];
#pragma unroll
      for (int q = 1; q < CL; ++q) m = fmaxf(m, u[q]);
      top = value_of(max8(key_of(m)));
      top = top > -INFINITY ? top : 0.f;
      sum = 0.f;
      if (by_logit) {
#pragma unroll
        for (int q = 0; q < CL; ++q) sum += fast_exp(u[q] - top);
      } else {                                          // (a masked expert is marked by -1)
#pragma unroll
        for (int q = 0; q < CL; ++q) {
          const float x = fast_exp(u[q] - top);
          sum += x;
          u[q] = !plain && !(u[q] > -INFINITY) ? -1.f : x;
        }
      }
      sum = sum8(sum);
    }
    const float inv = a.sigmoid ? 1.f : __fdividef(1.f, sum);
    // the keys, the lane's best eight in order; a place without an expert counts as a masked one
    uint32_t list[8] = {}, part[8];
    auto take = [&](int q, float v) {
      const uint32_t key = (key_of(v) & ~kIndex) | (index0 - q);
      if (q < 8) list[q & 7] = key;
      else part[q & 7] = key;
      if (q % 8 == 7 || q == CL - 1) {
        if (q < 8) {
          sort8(list);
        } else {
          sort8(part);
          merge8(list, part);
        }
      }
    };
    auto biased = [&](auto score) {
#pragma unroll
      for (int i = 0; i < CL; i += 4) {
        const float4 b = *reinterpret_cast<const float4*>(my_bias + i);
        take(i, score(u[i], b.x));
        take(i + 1, score(u[i + 1], b.y));
        take(i + 2, score(u[i + 2], b.z));
        take(i + 3, score(u[i + 3], b.w));
      }
    };
    if (by_logit) {
#pragma unroll
      for (int q = 0; q < CL; ++q) take(q, u[q]);
    } else if (!plain) {
      biased([&](float x, float b) {
        const float s = a.sigmoid ? __fdividef(1.f, 1.f + fast_exp(-x)) : x * inv;
        return (a.sigmoid ? x > -INFINITY : x >= 0.f) ? s + b : -INFINITY;
      });
    } else if (a.sigmoid) {
      biased([&](float x, float b) { return __fdividef(1.f, 1.f + fast_exp(-x)) + b; });
    } else {
      biased([&](float x, float b) { return x * inv + b; });
    }
    bool again = false;                                 // (the same in a token's lanes)
    if (GROUPED) {
      uint32_t g1 = list[0], g2 = list[1];
      for (int o = 1; o < a.seg; o <<= 1) {
        const uint32_t n1 = __shfl_xor_sync(kAll, g1, o), n2 = __shfl_xor_sync(kAll, g2, o);
        g2 = max(min(g1, n1), max(g2, n2));
        g1 = max(g1, n1);
      }
      const int own = sl >> a.seg_log;
      float mine = -INFINITY;
      if (own < a.groups) mine = a.group_top == 1 ? leading(g1) : leading(g1) + leading(g2);
      int better = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float v = __shfl_sync(kAll, mine, first + (g << a.seg_log));
        better += v > mine || (v == mine && g < own);
      }
      bool stays = own < a.groups && better < a.top_groups;
      if (a.top_groups < a.groups) {
        const float lo = -value_of(max8(stays ? key_of(-mine) : 0x007fffffu));   // (-inf)
        const float hi = value_of(max8(own < a.groups && !stays ? key_of(mine) : 0x007fffffu));
        // (a value is up to kLead of itself above its leading bits)
        const float most = bias_most + (a.sigmoid ? 1.f : inv);
        const float gap = by_logit ? 0.f : 2.f * near_of<CL>(a.sigmoid, inv, 2.f * most) + 2.f * kLead * most;
        again = hi > -INFINITY && !(lo - hi > gap || (by_logit && kLossless));
        if (a.seg == 1 && !by_logit && __any_sync(kAll, again)) {
          // a lane's own best: those of its first three by their fp32 values, if no other
          // comes near the last of them without being the same, and no other at all where one of the best does
          float x[3], bx[3], f[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const bool on = own < a.groups && leading(list[i]) > -INFINITY;
            const int q = (index0 - (list[i] & kIndex)) & (CL - 1);
            x[i] = on ? logit(a, row, e0 + q, &unused) : 0.f;
            bx[i] = on ? my_bias[q] : 0.f;
            f[i] = on ? score_of(a, x[i], top, inv) + bx[i] : -INFINITY;
          }
          auto order = [&](int i, int j) {
            if (!(f[j] > f[i])) return;
            const float t = f[i], tx = x[i], tb = bx[i];
            f[i] = f[j]; x[i] = x[j]; bx[i] = bx[j];
            f[j] = t; x[j] = tx; bx[j] = tb;
          };
          order(1, 2);
          order(0, 1);
          order(1, 2);
          const bool two = a.group_top == 2;
          const float least = two ? f[1] : f[0], xl = two ? x[1] : x[0], bl = two ? bx[1] : bx[0];
          const bool live = own < a.groups && least > -INFINITY;
          auto apart = [&](float hi, float lo, float lead) {
            return !(lo > -INFINITY) || hi - lo > near_of<CL>(a.sigmoid, inv, fmaxf(fabsf(hi), fabsf(lo))) + lead * fabsf(lo);
          };
          auto same = [&](int i) { return x[i] == xl && bx[i] == bl; };
          const bool third = apart(least, f[2], 0.f);
          bool unsure = live && !((two ? third || same(0) || apart(f[0], least, 0.f) : same(1) || apart(least, f[1], 0.f)) &&
                                  (third || same(2)) && apart(least, leading(list[3]), kLead));
          const Pair scale = a.sigmoid ? Pair{} : softmax_scales(a, row, top, __ballot_sync(kAll, again));
          const bool s = better_groups(a, x[0], bx[0], x[1], bx[1], live, own, first, 0, top, scale, &unsure);
          const unsigned open = __ballot_sync(kAll, unsure);
          if (again && !(open >> first & 0xffu)) {
            stays = s;
            again = false;
          }
        }
      }
      if (!stays) {
#pragma unroll
        for (int i = 0; i < 8; ++i) list[i] = 0;
      }
    }
    // the token's best eight, the same in all its lanes, and how the k-th compares to the next
    uint32_t best[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) best[i] = list[i];
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) part[i] = __shfl_xor_sync(kAll, best[i], o);
      merge8(best, part);
    }
    auto next_below = [&](uint32_t key) {               // (a lane's list ends with its eighth)
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, list[i] < key ? list[i] : 0u);
      return max8(m);
    };
    uint32_t sel = 0, kth = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (sl == i && i < a.k) sel = best[i];
      if (i == a.k - 1) kth = best[i];
    }
    const float last = leading(kth);
    int n = a.k, e = expert(sel);
    float l = sl < a.k ? logit(a, row, e, &unused) : -INFINITY;
    // (places without an expert count as masked ones: masked ones are chosen again)
    if (!(last > -INFINITY)) again = true;
    if (!(by_logit && kLossless) || __any_sync(kAll, again)) {
      // is it certain, and the order of neighbours?  By the fp32 values of the chosen, and by
      // the leading bits of the next
      uint32_t next = next_below(kth);
      float b = sl < a.k ? biases[e] : 0.f;
      const float v = !(l > -INFINITY) || by_logit ? l : score_of(a, l, top, inv) + b;
      const float kth_v = __shfl_sync(kAll, v, first + a.k - 1);
      auto certain = [&](uint32_t key, float than) {
        const float x = leading(key);
        if (!(x > -INFINITY) || by_logit) return !(x > -INFINITY) || last > x;
        return than - x > near_of<CL>(a.sigmoid, inv, fmaxf(fabsf(than), fabsf(x))) + kLead * fabsf(x);
      };
      // (a lane whose eight are all among the chosen may have a ninth: the token's lanes
      // look through that lane's experts once more, without those of its list.  One group
      // of 32 experts and 8 of them chosen, so that each token does: 30 us for 16384
      // instead of 23; 33 with that lane looking alone)
      const unsigned owns = __ballot_sync(kAll, list[7] >= kth && list[7] != 0) >> first & 0xffu;
      float ninth = -INFINITY;
      if (__any_sync(kAll, owns != 0)) {
        const int owner = owns ? __ffs(owns) - 1 : 0;
        uint32_t in_list = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) in_list |= 1u << ((index0 - list[i]) & (CL - 1));
        in_list = __shfl_sync(kAll, in_list, first + owner);
        if (owns) {
          const int from = first_of(owner), n_of = count_of(owner);
          for (int q = sl; q < n_of; q += 8) {
            const float x = logit(a, row, from + q, &unused);
            const float s = by_logit || !(x > -INFINITY) ? x : score_of(a, x, top, inv) + bias[owner * (CL + 4) + q];
            if (!(in_list >> q & 1)) ninth = fmaxf(ninth, s);
          }
        }
        ninth = value_of(max8(key_of(ninth)));
      }
      const float pv = __shfl_up_sync(kAll, v, 1, 8), pl = __shfl_up_sync(kAll, l, 1, 8), pb = __shfl_up_sync(kAll, b, 1, 8);
      const float gap = by_logit ? 0.f : near_pair<CL>(a.sigmoid, inv, pv, pb, v, b);
      const bool close = sl > 0 && v > -INFINITY && !(pv - v > gap) && !(pl == l && pb == b);
      const bool closes = __ballot_sync(kAll, close) >> first & 0xffu;
      const float than = closes ? last : kth_v;          // (the k-th only if their order is known)
      const bool full = ninth > -INFINITY &&
             !(than - ninth > (by_logit ? 0.f : near_of<CL>(a.sigmoid, inv, fmaxf(fabsf(than), fabsf(ninth)))));
      const bool sure = certain(next, than) && !full;
      if (__any_sync(kAll, closes || !sure || again)) {
        // more candidates, as long as one may be as good as the k-th
        uint32_t sel2 = 0, lowest = kth;
        for (int i = a.k; i < 16; ++i) {
          const bool more = !sure && !certain(next, last);
          if (!__any_sync(kAll, more)) break;
          if (more) {
            ++n;
            if (sl == i) sel = next;
            if (sl == i - 8) sel2 = next;
            lowest = next;
          }
          next = next_below(lowest);
        }
        // (16: there may be more; and a lane may have more than its list)
        const bool ended = __ballot_sync(kAll, list[7] >= lowest && list[7] != 0) >> first & 0xffu;
        bool open = again || n == 16 || (ended && (full || n > a.k));
        e = expert(sel);
        l = sl < n ? logit(a, row, e, &unused) : -INFINITY;
        b = sl < n ? biases[e] : 0.f;
        const int e2 = expert(sel2);
        const float l2 = sl + 8 < n ? logit(a, row, e2, &unused) : -INFINITY;
        const float b2 = sl + 8 < n ? biases[e2] : 0.f;
        e = order8<X, CL>(a, row, e, e2, l, l2, b, b2, n, top, inv, reinterpret_cast<int*>(slot));
        open = open || e < 0;
        const unsigned left = __ballot_sync(kAll, open);
        for (int o = 0; o < 32; o += 8)                  // what is left, a token at a time by the whole warp
          if (left >> o & 0xffu) {
            const X* r = reinterpret_cast<const X*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(row), o));
            const int x = choose32<X, (CL + 3) / 4, GROUPED>(a, r, slot);
            const int ex = __shfl_sync(kAll, x, sl);
            if (first == o) e = ex;
          }
        if (sl < a.k) l = logit(a, row, e, &unused);
      }
    }
    __syncwarp();                                       // (the slots are written again)
    if (sl >= a.k) l = -INFINITY;
    // gates, as above
    const bool none = !(__ballot_sync(kAll, l > -INFINITY) >> first & 0xffu);
    float w = !(l > -INFINITY) ? 0.f : a.sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - top);
    if (a.renorm) {
      const bool small = __ballot_sync(kAll, l > -INFINITY && l < -87.f) >> first & 0xffu;
      if (!a.sigmoid || __any_sync(kAll, small)) {
        const float x = a.sigmoid ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
        const float m = value_of(max8(key_of(x)));
        if (!a.sigmoid || small) w = l > -INFINITY ? expf(x - m) : 0.f;
      }
      w = w / sum8(w);
    } else if (!a.sigmoid) {
      w = w / sum;
    }
    if (none && mine_on) bad = true;
    if (mine_on && sl < a.k) {
      a.idx[t * a.k + sl] = e;
      a.gate[t * a.k + sl] = none ? 0.f : a.scale * w;
      atomicAdd(&hist[e], 1);
    }
  }
  if (bad) report(a.status, MOE_ERR_BAD_INPUT);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kManyThreads<CL>) a.hist[(int64_t)blockIdx.x * padded4(a.E) + e] = (uint16_t)hist[e];
}

// For at least kManyTokens per block; with fewer the longer way of a token through
// its lanes counts (256 experts in groups, us here / with a warp per token: 33 tokens per
// block 17.5 / 20, 20 tokens 16.5 / 15; 128 experts, 40 tokens 18.5 / 18.4).
constexpr int kManyTokens = 32;
template <typename X, int CL>
cudaError_t run_many(ScoreArgs a, int blocks, cudaStream_t s) {
  constexpr int kVec = CL * (int)sizeof(X) < 16 ? CL * (int)sizeof(X) : 16;
  // by vectors: rows and groups start on their boundaries
  a.vec = ((uintptr_t)a.logits & (kVec - 1)) == 0 && a.ld * sizeof(X) % kVec == 0 &&
          a.group_size * sizeof(X) % kVec == 0;
  return a.groups > 1 ? launch_overlapped(score_many_kernel<X, CL, true>, blocks, kManyThreads<CL>, 0, s, a)
                      : launch_overlapped(score_many_kernel<X, CL, false>, blocks, kManyThreads<CL>, 0, s, a);
}

}  // namespace

template <typename X>
cudaError_t launch_score_many(ScoreArgs a, int blocks, bool* taken, cudaStream_t s) {
  *taken = false;
  if (a.per_block < kManyTokens || blocks < 2 || a.k > 8 || a.groups > 8) return cudaSuccess;
  for (a.seg = 8, a.seg_log = 3; a.groups * a.seg > 8; a.seg /= 2) --a.seg_log;
  const int n = (a.group_size + a.seg - 1) / a.seg;      // experts of a lane
  if (n > 32) return cudaSuccess;
  *taken = true;
  return n <= 4 ? run_many<X, 4>(a, blocks, s)
         : n <= 8 ? run_many<X, 8>(a, blocks, s)
         : n <= 16 ? run_many<X, 16>(a, blocks, s)
                   : run_many<X, 32>(a, blocks, s);
}
template cudaError_t launch_score_many<float>(ScoreArgs, int, bool*, cudaStream_t);
template cudaError_t launch_score_many<__nv_bfloat16>(ScoreArgs, int, bool*, cudaStream_t);

}  // namespace moe
