// score_route.cuh - what the two kernels of the router by scores share
// (score_route.cu: a warp per token; score_many.cu: eight lanes per token): scores and
// their errors, the order of close values, the choice from all bits by a whole warp.
#pragma once

#include "rows.cuh"

namespace moe {

__host__ __device__ __forceinline__ int padded4(int E) { return (E + 3) & ~3; }

struct ScoreArgs {
  const void* logits;
  const float* bias;
  int64_t ld;
  int T, E, k, per_block;
  int groups, group_size, top_groups, group_top;
  int seg, seg_log;         // lanes of a group where it has 2^seg_log, else 0
  int sigmoid, renorm, vec;
  float scale;
  int32_t* idx;
  float* gate;
  uint16_t* hist;           // [blocks][padded4(E)]
  int32_t* status;
};

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

// exp(x) by one MUFU instruction: relative error below 2^-22 + 1.4 |x| 2^-24.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504088896341f));
  return r;
}

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

// A lane's C neighbouring logits of a row as they lie in memory: by vectors of up
// to 16 bytes, where rows start on their boundaries and E is whole vectors, else by
// elements.
template <typename X, int C>
struct Logits {
  static constexpr int kBytes = C * (int)sizeof(X), kVec = kBytes < 16 ? kBytes : 16;
  static constexpr int N = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[N];
  __device__ __forceinline__ void load(const X* row, int E, bool vec) {
    const int e0 = (threadIdx.x & 31) * C;
    if (vec && kBytes >= 4) {
#pragma unroll
      for (int i = 0; i < kBytes / kVec; ++i) {
        if (e0 + i * (kVec / (int)sizeof(X)) >= E) continue;
        const X* p = row + e0 + i * (kVec / (int)sizeof(X));
        if constexpr (kVec == 16) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        } else if constexpr (kVec == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[0] = v.x; w[N - 1] = v.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < C; ++q) {
        if (e0 + q >= E) continue;
        if constexpr (sizeof(X) == 4) {
          w[q] = __float_as_uint(row[e0 + q]);
        } else {
          const uint32_t v = __bfloat16_as_ushort(row[e0 + q]);
          w[q / 2] = q & 1 ? (w[q / 2] & 0xffffu) | v << 16 : v;
        }
      }
    }
  }
  __device__ __forceinline__ float get(int q) const {
    return sizeof(X) == 4 ? __uint_as_float(w[q % N]) : q & 1 ? bf16_hi(w[(q / 2) % N]) : bf16_lo(w[(q / 2) % N]);
  }
};

// Largest distance of two fp32 values u that may be in the other order (or
// equal) in 64 bits; `s` bounds the scores (1, or the largest of the softmax), `u`
// the values.  In units of 2^-24: fast_exp is off by 4 + 1.4 |x| relative to its value.
// Sigmoid: that enters as s (1 - s), at most 1 + 0.3; 1 + exp rounds by 1, the
// reciprocal by 2, the bias' addition by |u|: below 5 + |u| each.  Softmax, relative to
// the largest score: 4 + 0.9 of the exponential (its argument rounds too), 4 + 2.4 ln E of
// the sum's terms, C + 4 of their addition, 3 of the quotient: below 32 + C.
template <int C>
__device__ __forceinline__ float near_of(bool sigmoid, float s, float u) {
  return (sigmoid ? 10 * 0x1p-24f : (64 + 2 * C) * 0x1p-24f * s) + 0x1p-23f * fabsf(u);
}

// The same for two values (u, b) and (v, c) whose biases are known.  The softmax' sum
// is off by 28 + C for both alike, which moves their scores' difference, at most that of
// the biases and their own, by as much relative to it; 7 relative to each score and 1.8
// to the largest are their own.
template <int C>
__device__ __forceinline__ float near_pair(bool sigmoid, float s, float u, float b, float v, float c) {
  const float w = fmaxf(fabsf(u), fabsf(v));
  if (sigmoid) return near_of<C>(true, 1.f, w);
  return 0x1p-24f * ((30 + C) * (fabsf(b - c) + fabsf(u - v)) + 7.5f * (fabsf(u - b) + fabsf(v - c)) + 2.f * s) +
         0x1p-23f * w;
}

// The best two keys of a lane with their places (of equal ones the first).
template <int C>
struct BestTwo {
  uint32_t m1, m2;
  int q1, q2;
  __device__ __forceinline__ void take(const uint32_t (&key)[C]) {
    m1 = key[0];
    q1 = 0;
    m2 = 0;
    q2 = 0;
#pragma unroll
    for (int q = 1; q < C; ++q) {
      const bool a = key[q] > m1, b = key[q] > m2;
      m2 = a ? m1 : b ? key[q] : m2;
      q2 = a ? q1 : b ? q : q2;
      m1 = a ? key[q] : m1;
      q1 = a ? q : q1;
    }
  }
  // takes the best away; the next after the second is looked for again
  __device__ __forceinline__ void pop(const uint32_t (&key)[C]) {
    const uint32_t last = m1;
    const int at = q1;
    m1 = m2;
    q1 = q2;
    m2 = 0;
    if (m1 == 0) {
#pragma unroll
      for (int q = C - 1; q >= 0; --q)
        if ((key[q] < last || (key[q] == last && q > at)) && key[q] >= m1) {
          m1 = key[q];
          q1 = q;
        }
    }
  }
};

// ------------------------------------------------- pairs of fp32 numbers
// h + l with |l| at most half a unit of h: 46 to 48 significant bits from fp32
// instructions (the sums and products of Dekker and Knuth), for the values that fp32
// cannot order.  (fp64 took 7 to 9 us for two values and 43 for a row of 256.)
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair normal(float h, float l) {            // |h| >= |l|
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = sum_of(a.h, b.h), t = sum_of(a.l, b.l);
  const Pair u = normal(s.h, __fadd_rn(s.l, t.h));
  return normal(u.h, __fadd_rn(u.l, t.l));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);
  float e = __fmaf_rn(a.h, b.h, -p);
  e = __fmaf_rn(a.h, b.l, e);
  e = __fmaf_rn(a.l, b.h, e);
  return normal(p, e);
}
__device__ __forceinline__ Pair inverse(Pair d) {
  const float y = __frcp_rn(d.h);
  const float e = __fmaf_rn(-d.l, y, __fmaf_rn(-d.h, y, 1.f));
  return normal(y, __fmul_rn(y, e));
}
// exp(x), -80 <= x <= 0, relative error below 2^-40: x - n ln 2 (ln 2 in three parts,
// the first of 15 bits, so that its product with n is exact), a 16th of that in the
// Taylor series up to the 7th power (the rest is below 2^-59), squared four times.
__device__ __forceinline__ Pair exp_of(Pair x) {
  const float n = rintf(x.h * 1.44269504f);
  Pair r = sum_of(x.h, -n * 0x1.62e4p-1f);
  r = add(r, {x.l, 0.f});
  const float p = __fmul_rn(n, -0x1.7f7d1cp-20f), pe = __fmaf_rn(n, -0x1.7f7d1cp-20f, -p);
  r = add(r, normal(p, __fmaf_rn(n, -0x1.ef357ap-45f, pe)));
  r.h *= 0.0625f;
  r.l *= 0.0625f;
  const float t = fmaf(fmaf(1.f / 5040, r.h, 1.f / 720), r.h, 1.f / 120);
  Pair y = normal(0x1.555556p-5f, fmaf(r.h, t, -0x1.555556p-30f));    // 1/24 + ...
  y = add(mul(y, r), {0x1.555556p-3f, -0x1.555556p-28f});              // 1/6
  y = add(mul(y, r), {0.5f, 0.f});
  y = add(mul(y, r), {1.f, 0.f});
  y = add(mul(y, r), {1.f, 0.f});
#pragma unroll
  for (int i = 0; i < 4; ++i) y = mul(y, y);
  const float f = __uint_as_float((uint32_t)(127 + (int)n) << 23);     // n >= -116
  return {y.h * f, y.l * f};
}
// What a candidate is compared by: its value, and how far off that may be.
struct Exact {
  Pair u;
  float off;                // infinite: not known to this precision
};
__device__ __forceinline__ Exact exact_of(float s_h, float s_l, float b, bool known) {
  const Pair t = sum_of(s_h, b);
  const Pair u = normal(t.h, __fadd_rn(t.l, s_l));
  return {u, known ? 0x1p-39f * s_h + 0x1p-44f * fabsf(u.h) : INFINITY};
}

// A token's softmax (largest logit and sum of exponentials relative to it); u:
// this lane's logits.
template <int C>
__device__ __forceinline__ void softmax_of(const float (&u)[C], float* top, float* sum) {
  float m = u[0];
#pragma unroll
  for (int q = 1; q < C; ++q) m = fmaxf(m, u[q]);
  m = value_of(__reduce_max_sync(kAll, key_of(m)));
  m = m > -INFINITY ? m : 0.f;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < C; ++q) s += fast_exp(u[q] - m);
  *top = m;
  *sum = warp_sum(s);
}
__device__ __forceinline__ float score_of(const ScoreArgs& a, float l, float top, float inv_sum) {
  return a.sigmoid ? __fdividef(1.f, 1.f + fast_exp(-l)) : fast_exp(l - top) * inv_sum;
}

// 1 / (the sum of this row's exponentials relative to top), by a whole warp.
template <typename X>
__device__ __noinline__ Pair softmax_scale(const ScoreArgs& a, const X* row, float top) {
  Pair sum{0.f, 0.f};
  bool bad = false;
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < a.E; e += 32) {
    const Pair x = sum_of(logit(a, row, e, &bad), -top);
    if (x.h > -80.f) sum = add(sum, exp_of(x));
  }
#pragma unroll 1
  for (int o = 16; o; o >>= 1) sum = add(sum, {__shfl_xor_sync(kAll, sum.h, o), __shfl_xor_sync(kAll, sum.l, o)});
  return inverse(sum);
}

// u of one candidate of each lane (logit l, bias b; a softmax' largest logit and scale).
__device__ __noinline__ Exact exact_value(bool sigmoid, float l, float b, float top, Pair scale) {
  const Pair x = sigmoid ? Pair{-fabsf(l), 0.f} : sum_of(l, -top);
  const bool known = x.h > -80.f;
  const Pair e = exp_of(known ? x : Pair{-80.f, 0.f});
  const Pair inv = sigmoid ? inverse(add({1.f, 0.f}, e)) : scale;
  const Pair s = sigmoid && l >= 0.f ? inv : mul(e, inv);
  return exact_of(s.h, s.l, b, known);
}

// The order of n candidates, one per lane (expert e, logit l, bias b): from fp32, and
// where that does not tell from pairs of it.  Returns the lane's expert in that order;
// -1 to all lanes if pairs do not tell either.
template <typename X, int C>
__device__ __noinline__ int order(const ScoreArgs& a, const X* row, int e, float l, float b, int n, float top, float inv,
                                  uint2* slot) {
  const int lane = threadIdx.x & 31;
  const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
  const bool on = lane < n && l > -INFINITY;
  const float v = !on || by_logit ? l : score_of(a, l, top, inv) + b;
  int better = 0;
  bool unsure = false;
  for (int i = 0; i < n; ++i) {
    const float ov = __shfl_sync(kAll, v, i), ol = __shfl_sync(kAll, l, i), ob = __shfl_sync(kAll, b, i);
    const int oe = __shfl_sync(kAll, e, i);
    const bool other = ol > -INFINITY;
    const float gap = by_logit ? 0.f : near_pair<C>(a.sigmoid, inv, v, b, ov, ob);
    if (oe == e) continue;
    if ((ol == l && ob == b) || (!on && !other)) better += oe < e;
    else if (!on || !other) better += other;               // masked ones last
    else if (fabsf(ov - v) > gap || by_logit) better += ov > v || (ov == v && oe < e);
    else unsure = true;
  }
  if (__any_sync(kAll, lane < n && unsure)) {
    const Exact x = exact_value(a.sigmoid, l, b, top, a.sigmoid ? Pair{} : softmax_scale(a, row, top));
    better = 0;
    unsure = false;
    for (int i = 0; i < n; ++i) {
      const float oh = __shfl_sync(kAll, x.u.h, i), olow = __shfl_sync(kAll, x.u.l, i);
      const float off = __shfl_sync(kAll, x.off, i) + x.off;
      const float ol = __shfl_sync(kAll, l, i), ob = __shfl_sync(kAll, b, i);
      const int oe = __shfl_sync(kAll, e, i);
      const bool other = ol > -INFINITY;
      if (oe == e) continue;
      const float d = (oh - x.u.h) + (olow - x.u.l);
      if ((ol == l && ob == b) || (!on && !other)) better += oe < e;
      else if (!on || !other) better += other;
      else if (fabsf(d) > off) better += d > 0.f;
      else unsure = true;
    }
    if (__any_sync(kAll, lane < n && unsure)) return -1;
  }
  __syncwarp();
  if (lane < n) slot[better].y = e;
  __syncwarp();
  return lane < n ? slot[lane].y : 0;
}

// Whether this lane's group `own` is among the best: l0, b0, l1, b1 are logits and
// biases of its best one or two (live: none masked), lane base + (g << log) has group
// g's.  *unsure: whether these do not tell.
__device__ __noinline__ bool better_groups(const ScoreArgs& a, float l0, float b0, float l1, float b1, bool live, int own,
                                           int base, int log, float top, Pair scale, bool* unsure) {
  if (!live) l0 = b0 = 0.f;
  if (!live || a.group_top == 1) l1 = b1 = 0.f;
  const Exact x0 = exact_value(a.sigmoid, l0, b0, top, scale), x1 = exact_value(a.sigmoid, l1, b1, top, scale);
  Pair mine = x0.u;
  float off = x0.off;
  if (a.group_top == 2) {
    mine = add(x0.u, x1.u);
    off += x1.off + 0x1p-44f * (fabsf(x0.u.h) + fabsf(x1.u.h));
  }
  int better = 0;
  for (int g = 0; g < a.groups; ++g) {
    // (every lane takes part in every exchange: none of them behind a condition)
    const int at = base + (g << log);
    const bool ol = __shfl_sync(kAll, (int)live, at);
    const float oh = __shfl_sync(kAll, mine.h, at), olow = __shfl_sync(kAll, mine.l, at);
    const float oo = __shfl_sync(kAll, off, at) + off;
    const float m0 = __shfl_sync(kAll, l0, at), m1 = __shfl_sync(kAll, l1, at);
    const float n0 = __shfl_sync(kAll, b0, at), n1 = __shfl_sync(kAll, b1, at);
    const bool same = m0 == l0 && m1 == l1 && n0 == b0 && n1 == b1;
    if (g == own || own >= a.groups) continue;
    const float d = (oh - mine.h) + (olow - mine.l);
    if (!ol || !live) better += ol != live ? ol : g < own;
    else if (same) better += g < own;
    else if (fabsf(d) > oo) better += d > 0.f;
    else *unsure = true;
  }
  return own < a.groups && better < a.top_groups;
}

// Which groups stay (lane g: group g), from the values of their best in pairs of
// fp32; *sure: whether these tell.
template <typename X, int C>
__device__ __noinline__ bool exact_groups(const ScoreArgs& a, const X* row, const uint32_t (&key)[C],
                                          float top, float inv, bool* sure) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  bool bad = false;
  float worst = -INFINITY, lg[2] = {}, bg[2] = {};         // lane g: its group's best one or two, the last of them by value
  uint32_t won = 0;                                        // this lane's experts among these
  for (int g = 0; g < a.groups; ++g) {
    for (int r = 0; r < a.group_top; ++r) {
      uint32_t m = 0;
      int at = 0;
#pragma unroll
      for (int q = C - 1; q >= 0; --q) {
        const int x = lane * C + q;
        if (x >= g * a.group_size && x < (g + 1) * a.group_size && !(won >> q & 1u) && key[q] >= m && key[q]) {
          m = key[q];
          at = q;
        }
      }
      const uint32_t f = __reduce_max_sync(kAll, m);
      const unsigned who = __ballot_sync(kAll, m == f && f);
      const bool win = (who >> lane & 1u) && !(who & below);
      if (win) won |= 1u << at;
      const int x = __shfl_sync(kAll, lane * C + at, who ? __ffs(who) - 1 : 0);
      if (lane == g) {
        const float lx = f ? logit(a, row, x, &bad) : -INFINITY, bx = f ? bias_of(a, x) : 0.f;
        worst = f ? value_of(f) : -INFINITY;
        if (r == 0) { lg[0] = lx; bg[0] = bx; }
        else { lg[1] = lx; bg[1] = bx; }
      }
    }
  }
  // Which are the best is certain if no other one comes close to the last of them, or if all
  // that do, among the best too, are the same as it.  (Next to twins of it, a close one may lie
  // above them that fp32 has below, or below them that it has among the best.)
  const float lk = a.group_top == 1 ? lg[0] : lg[1], bk = a.group_top == 1 ? bg[0] : bg[1];
  uint32_t more = 0, mixed = 0;                            // by group
#pragma unroll 4
  for (int q = 0; q < C; ++q) {
    const int x = lane * C + q, g = min(x / a.group_size, a.groups - 1);
    const float last = __shfl_sync(kAll, worst, g), ll = __shfl_sync(kAll, lk, g), bl = __shfl_sync(kAll, bk, g);
    const float w = key[q] ? value_of(key[q]) : -INFINITY;
    if (last > -INFINITY && w > -INFINITY && !(fabsf(last - w) > near_of<C>(a.sigmoid, inv, fmaxf(fabsf(last), fabsf(w))))) {
      if (!(won >> q & 1u)) more |= 1u << g;
      if (!(logit(a, row, x, &bad) == ll && bias_of(a, x) == bl)) mixed |= 1u << g;
    }
  }
  bool unsure = (__reduce_or_sync(kAll, more) & __reduce_or_sync(kAll, mixed)) >> lane & 1u;
  const bool live = lane < a.groups && worst > -INFINITY;    // (a group with a masked one among its best counts as -inf)
  const bool stays = better_groups(a, lg[0], bg[0], lg[1], bg[1], live, lane, 0, 0, top,
                                   a.sigmoid ? Pair{} : softmax_scale(a, row, top), &unsure);
  *sure = !__any_sync(kAll, unsure);
  return stays;
}

// The choice for one token from all bits of its values: rounds of a warp maximum
// over (value, lower index).  Values that fp32 cannot order are taken in pairs of it:
// those of the candidates, which are the k chosen and all that come close to the
// last of them.
template <typename X, int C, bool GROUPED>
__device__ __noinline__ int choose32(const ScoreArgs& a, const X* row, uint2* slot) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  const bool by_logit = !a.bias && (!GROUPED || a.group_top == 1);
  bool bad = false;
  float u[C], top = 0.f, sum = 1.f;
#pragma unroll
  for (int q = 0; q < C; ++q) u[q] = lane * C + q < a.E ? logit(a, row, lane * C + q, &bad) : -INFINITY;
  if (!a.sigmoid && !by_logit) softmax_of(u, &top, &sum);
  const float inv = 1.f / sum;
  uint32_t key[C];
#pragma unroll
  for (int q = 0; q < C; ++q) {
    const int e = lane * C + q;
    key[q] = e >= a.E ? 0 : key_of(by_logit || !(u[q] > -INFINITY) ? u[q] : score_of(a, u[q], top, inv) + bias_of(a, e));
  }
  if (GROUPED) {
    float mine = -INFINITY;              // lane g: the value of group g
    uint32_t part = 0;                   // the largest of its addends
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
      const uint32_t b1 = __reduce_max_sync(kAll, m1);
      float v = value_of(b1), x = fabsf(v);
      if (a.group_top > 1) {
        const unsigned who = __ballot_sync(kAll, m1 == b1);
        const float second = value_of(__reduce_max_sync(kAll, lane == __ffs(who) - 1 ? m2 : m1));
        v += second;
        x = fmaxf(x, fabsf(second));
      }
      if (lane == g) {
        mine = v;
        part = __float_as_uint(x < INFINITY ? x : 0.f);
      }
    }
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float v = __shfl_sync(kAll, mine, g);
      better += v > mine || (v == mine && g < lane);
    }
    bool stays = lane < a.groups && better < a.top_groups, sure = true;
    if (!by_logit && a.top_groups < a.groups) {
      const float lo = -value_of(__reduce_max_sync(kAll, stays ? key_of(-mine) : 0x007fffffu));   // (-inf)
      const float hi = value_of(__reduce_max_sync(kAll, lane < a.groups && !stays ? key_of(mine) : 0x007fffffu));
      const float big = __uint_as_float(__reduce_max_sync(kAll, part));
      if (hi > -INFINITY && !(lo - hi > 2.f * near_of<C>(a.sigmoid, inv, 2.f * big))) {
        stays = exact_groups<X, C>(a, row, key, top, inv, &sure);
        if (!sure) return choose64<X, C>(a, row);
      }
    }
    const unsigned stay = __ballot_sync(kAll, stays);
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const int e = lane * C + q;
      if (e < a.E && !(stay >> (e / a.group_size) & 1u)) key[q] = 0;
    }
  }
  BestTwo<C> best;
  best.take(key);
  // (a lane with nothing left has 0 and wins nothing, as long as others have some)
  float last = -INFINITY;                  // the k-th value
  int n = 0;
  for (; n < 32; ++n) {
    const uint32_t m = __reduce_max_sync(kAll, best.m1);
    if (n >= a.k) {
      const float v = m ? value_of(m) : -INFINITY;
      if (by_logit || !(v > -INFINITY) || last - v > near_of<C>(a.sigmoid, inv, fmaxf(fabsf(last), fabsf(v)))) break;
    }
    const bool eq = best.m1 == m;
    if (!(__ballot_sync(kAll, eq) & below) && eq) {
      slot[n] = make_uint2(m, lane * C + best.q1);
      best.pop(key);
    }
    if (n == a.k - 1) last = value_of(m);
    __syncwarp();
  }
  __syncwarp();
  const uint2 sel = lane < n ? slot[lane] : make_uint2(0, 0);
  int sel_e = sel.y;
  if (by_logit) return sel_e;
  bool unused = false;
  const float l = sel.x ? logit(a, row, sel_e, &unused) : -INFINITY, b = sel.x ? bias_of(a, sel_e) : 0.f;
  // (with all places taken others may be as close: known only if all that come close to the
  // k-th, candidates or not, are the same as it, so that their order is that of their indices)
  bool more = false;
  if (n == 32) {
    const float lk = __shfl_sync(kAll, l, a.k - 1), bk = __shfl_sync(kAll, b, a.k - 1);
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const float w = key[q] ? value_of(key[q]) : -INFINITY;
      if (w > -INFINITY && !(fabsf(last - w) > near_of<C>(a.sigmoid, inv, fmaxf(fabsf(last), fabsf(w)))) &&
          !(u[q] == lk && bias_of(a, lane * C + q) == bk))
        more = true;
    }
  }
  if (__any_sync(kAll, more)) return choose64<X, C>(a, row);
  const int e = order<X, C>(a, row, sel_e, l, b, n, top, inv, slot);
  return __any_sync(kAll, e < 0) ? choose64<X, C>(a, row) : e;
}

}  // namespace

// Where a token count is large and the sizes fit: the choice, gates and
// histograms by eight lanes per token; *taken: whether they did.
template <typename X>
cudaError_t launch_score_many(ScoreArgs a, int blocks, bool* taken, cudaStream_t s);

}  // namespace moe
