// score_route.cu - routing by scores: softmax or sigmoid scores, a bias for
// balance, groups of experts, top-k, gates; its backward; the bias' update.
//
//   s = softmax(l) or 1 / (1 + exp(-l)),  u = s + bias
//   a group's value is the sum of its `group_top` largest u; the `top_groups`
//   best groups stay; the k largest u in them are chosen (ties: the lower
//   index), and gate_j = scale s_j, or scale s_j / sum of the chosen s.
//
// The choice is that of u in 64 bits, whatever the GPU, found in three steps:
//   - keys of 32 bits that hold the leading bits of u in fp32 and the expert's
//     index, all different, so that a round of the choice is one warp maximum
//     (about 250 instructions a token where comparing values and indices took 750);
//   - where two values that the choice turns on are not told apart by these bits and
//     the error of fp32 (near_of): the token's values in full fp32, and those that
//     are still too close as pairs of fp32 numbers (choose32);
//   - where more than a warp's worth of values are too close, or pairs of fp32 numbers
//     do not tell: all of the token in 64 bits (choose64).  fp64 for every value would
//     take 30 times the time that the logits take from HBM.
// Without a bias u orders as the logits do, which are compared themselves.
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

// exp(x) by one MUFU instruction: relative error below 2^-22 + 1.4 |x| 2^-24.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504088896341f));
  return r;
}

__host__ __device__ __forceinline__ int padded4(int E) { return (E + 3) & ~3; }

struct ScoreArgs {
  const void* logits;
  const float* bias;
  int64_t ld;
  int T, E, k, per_block;
  int groups, group_size, top_groups, group_top;
  int seg, seg_log;         // lanes of a group where it is 2^seg_log whole lanes, else 0
  int sigmoid, renorm, vec;
  float scale;
  int32_t* idx;
  float* gate;
  int32_t* hist;            // [blocks][padded4(E)]
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
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        } else if constexpr (kVec == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
          w[0] = v.x; w[N - 1] = v.y;
        } else {
          w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
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
    const float gap = by_logit ? 0.f : near_of<C>(a.sigmoid, inv, fmaxf(fabsf(v), fabsf(ov)));
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
  float v[3] = {-INFINITY, -INFINITY, -INFINITY};          // lane g: its best three, the last known by value
  float lg[3] = {}, bg[3] = {};
  for (int g = 0; g < a.groups; ++g) {
    uint32_t gone = 0;
    for (int r = 0; r <= a.group_top; ++r) {
      uint32_t m = 0;
      int at = 0;
#pragma unroll
      for (int q = C - 1; q >= 0; --q) {
        const int x = lane * C + q;
        if (x >= g * a.group_size && x < (g + 1) * a.group_size && !(gone >> q & 1u) && key[q] >= m && key[q]) {
          m = key[q];
          at = q;
        }
      }
      const uint32_t f = __reduce_max_sync(kAll, m);
      const unsigned who = __ballot_sync(kAll, m == f && f);
      const bool win = (who >> lane & 1u) && !(who & below);
      if (win) gone |= 1u << at;
      const int x = __shfl_sync(kAll, lane * C + at, who ? __ffs(who) - 1 : 0);
      if (lane == g) {
        const float lx = f ? logit(a, row, x, &bad) : -INFINITY, bx = f ? bias_of(a, x) : 0.f;
        if (r == 0) { v[0] = f ? value_of(f) : -INFINITY; lg[0] = lx; bg[0] = bx; }
        else if (r == 1) { v[1] = f ? value_of(f) : -INFINITY; lg[1] = lx; bg[1] = bx; }
        else { v[2] = f ? value_of(f) : -INFINITY; lg[2] = lx; bg[2] = bx; }
      }
    }
  }
  // the group's best are certain if the next one lies apart or is the same
  const int t = a.group_top;
  const float last = t == 1 ? v[0] : v[1], next = t == 1 ? v[1] : v[2];
  const float ll = t == 1 ? lg[0] : lg[1], bl = t == 1 ? bg[0] : bg[1], ln = t == 1 ? lg[1] : lg[2], bn = t == 1 ? bg[1] : bg[2];
  bool unsure = lane < a.groups && next > -INFINITY && !(last - next > near_of<C>(a.sigmoid, inv, fmaxf(fabsf(last), fabsf(next)))) &&
                !(ll == ln && bl == bn);
  const bool live = lane < a.groups && last > -INFINITY;     // (a group with a masked one among its best counts as -inf)
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
  bool more = false;                       // close ones that found no place among the candidates
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

// Rows of the tokens [t0, t1) of one block: run[e] is the row of expert e's next
// assignment.  A token chooses an expert at most once, so the rank of an
// assignment is the number of earlier tokens with the same expert: a bit per token
// and expert, set in any order, counted up to the token's own.
struct PlaceArgs {
  const int32_t* idx;
  const int32_t* hist;       // [nb][padded4(E)]
  int T, k, E, nb, per_block, words;
  int64_t max_rows, sure;    // rows at or past `sure` belong to no expert, whatever the routing
  int32_t* counts;
  int32_t* offsets;
  int32_t* padded;
  int32_t* row_of;
  int32_t* assign_of;
};

__device__ __forceinline__ void place_tokens(const PlaceArgs& a, int64_t t0, int64_t t1, int* run, uint32_t* bits) {
  const int round = 32 * a.words;
  for (int64_t base = t0; base < t1; base += round) {
    const int n = (int)min((int64_t)round, t1 - base), words = (n + 31) >> 5;
    for (int i = threadIdx.x; i < words * a.E; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    const int32_t* idx = a.idx + base * a.k;
    for (int i = threadIdx.x; i < n * a.k; i += blockDim.x) {
      const int t = i / a.k;
      atomicOr(&bits[(t >> 5) * a.E + idx[i]], 1u << (t & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * a.k; i += blockDim.x) {
      const int t = i / a.k, e = idx[i];
      int row = run[e];
      for (int w = 0; w < t >> 5; ++w) row += __popc(bits[w * a.E + e]);
      row += __popc(bits[(t >> 5) * a.E + e] & ((1u << (t & 31)) - 1u));
      a.row_of[base * a.k + i] = row;
      a.assign_of[row] = (int)(base * a.k + i);
    }
    __syncthreads();
    if (base + round < t1) {
      for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        for (int w = 0; w < words; ++w) run[e] += __popc(bits[w * a.E + e]);
      __syncthreads();
    }
  }
}

// Exclusive sums over the experts of their counts and of these rounded up to
// kAlign: off and start [E + 1] in shared memory, by the whole block (sm: 32).
__device__ __forceinline__ void scan_experts(const int* cnt, int E, int* off, int* start, int2* sm) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int2 before = make_int2(0, 0);
  for (int c0 = 0; c0 < E; c0 += blockDim.x) {
    const int used = (min(E - c0, (int)blockDim.x) + 31) >> 5;        // warps with experts
    const int e = c0 + threadIdx.x, n = e < E ? cnt[e] : 0, p = (n + kAlign - 1) / kAlign * kAlign;
    int x = n, y = p;
    if (w < used) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kAll, x, o), v = __shfl_up_sync(kAll, y, o);
        if (lane >= o) {
          x += u;
          y += v;
        }
      }
      if (lane == 31) sm[w] = make_int2(x, y);
    }
    __syncthreads();
    if (w < used) {
      int2 all = lane < used ? sm[lane] : make_int2(0, 0), mine = lane < w ? all : make_int2(0, 0);
      all.x = __reduce_add_sync(kAll, all.x);
      all.y = __reduce_add_sync(kAll, all.y);
      mine.x = __reduce_add_sync(kAll, mine.x);
      mine.y = __reduce_add_sync(kAll, mine.y);
      if (e < E) {
        off[e] = before.x + mine.x + x - n;
        start[e] = before.y + mine.y + y - p;
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

// Rows without an assignment up to row `end`: those behind each expert's, and behind the last.
__device__ __forceinline__ void fill_rows(const PlaceArgs& a, const int* cnt, const int* start, int64_t end, int b,
                                          int nb) {
  const int w = threadIdx.x >> 5, nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  for (int e = b * nw + w; e < a.E; e += nb * nw)
    for (int r = start[e] + cnt[e] + lane; r < start[e + 1]; r += 32) a.assign_of[r] = -1;
  no_assignment(a, start[a.E], end, b, nb);
}

// Threads of a block at most: the keys of wider rows take more registers.
template <int C>
constexpr int kRouteThreads = C <= 4 ? 1024 : C <= 8 ? 768 : C <= 16 ? 512 : 256;

// FUSED: the first block has all tokens (few of them) and places them too,
// without a second launch; the others fill the rows from p.sure on, which no routing reaches.
template <typename X, int C, bool GROUPED, bool FUSED>
__global__ void __launch_bounds__(kRouteThreads<C>) score_route_kernel(const __grid_constant__ ScoreArgs a,
                                                           const __grid_constant__ PlaceArgs p) {
  __shared__ int hist[kMaxE];
  __shared__ uint2 slots[32][33];
  __shared__ int2 scan[32];
  extern __shared__ uint32_t dyn[];
  let_next_start();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  wait_for_previous();
  if (FUSED && blockIdx.x > 0) {
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
  Logits<X, C> next;
  if (t < t1) next.load(static_cast<const X*>(a.logits) + t * a.ld, a.E, a.vec);
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
      const float gap = by_logit ? 0.f : near_of<C>(a.sigmoid, inv, fmaxf(fabsf(pv), fabsf(v))) + kLead * fabsf(v);
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
      // relative to the largest chosen score where sigmoids are small (their sum may be 0), and for the softmax
      if (!a.sigmoid || !__any_sync(kAll, l > -60.f)) {
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
      a.gate[t * a.k + lane] = none ? 0.f : a.scale * w;
      atomicAdd(&hist[sel_e], 1);
    }
  }
  if (bad) report(a.status, MOE_ERR_BAD_INPUT);
  __syncthreads();
  if constexpr (FUSED) {
    int* off = reinterpret_cast<int*>(dyn);
    int* start = off + a.E + 1;
    int* run = start + a.E + 1;
    scan_experts(hist, a.E, off, start, scan);
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
      if (e < a.E) {
        run[e] = start[e];
        p.counts[e] = hist[e];
      }
      p.offsets[e] = off[e];
      p.padded[e] = start[e];
    }
    __syncthreads();
    place_tokens(p, 0, a.T, run, reinterpret_cast<uint32_t*>(run + a.E));
    fill_rows(p, hist, start, gridDim.x > 1 ? p.sure : p.max_rows, 0, 1);
  } else {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * padded4(a.E) + e] = hist[e];
  }
}

// Many tokens: eight lanes per token, four tokens per warp, so that what a token
// takes besides its elements (rounds, gates, addresses) is paid once for four.
// E <= 8 CL, top_k <= 8, a group is a power of two of lanes or all there is; rows by
// vectors.  Of fp32 logits a key's index is that within the lane, which leaves more bits
// to the value.
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
      const float gap = near_of<CL>(a.sigmoid, inv, fmaxf(fabsf(v[r]), fabsf(ov)));
      if ((ol == l[r] && ob == b[r]) || (!on[r] && !other)) better[r] += oe < e[r];
      else if (!on[r] || !other) better[r] += other;               // masked ones last
      else if (by_logit || fabsf(ov - v[r]) > gap) better[r] += ov > v[r] || (ov == v[r] && oe < e[r]);
      else unsure = true;
    }
  }
  unsigned open = __ballot_sync(kAll, unsure);
  if (open) {
    Pair scale{};
    if (!a.sigmoid) {
      for (int t = 0; t < 32; t += 8)                        // a token at a time, by the whole warp
        if (open >> t & 0xffu) {
          const X* r = reinterpret_cast<const X*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(row), t));
          const Pair p = softmax_scale(a, r, __shfl_sync(kAll, top, t));
          if (first == t) scale = p;
        }
    }
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
        const float gap = near_of<CL>(a.sigmoid, inv, fmaxf(fabsf(v[r]), fabsf(ov)));
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

// A lane's best keys, the largest first (more are looked for again when these are
// taken: 0.6 times a token with three of 16 kept, with four of 32 and half of the groups gone).
template <int CL>
struct BestKeys {
  static constexpr int K = CL > 16 ? 4 : 3;
  uint32_t m[K];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < K; ++i) m[i] = 0;
  }
  __device__ __forceinline__ void insert(uint32_t k) {
#pragma unroll
    for (int i = K - 1; i > 0; --i) m[i] = max(m[i], min(m[i - 1], k));
    m[0] = max(m[0], k);
  }
  __device__ __forceinline__ void pop(const uint32_t (&key)[CL]) {
    const uint32_t last = m[0];
#pragma unroll
    for (int i = 0; i + 1 < K; ++i) m[i] = m[i + 1];
    m[K - 1] = 0;
    if (m[0] == 0) {
#pragma unroll
      for (int q = 0; q < CL; ++q)
        if (key[q] < last) m[0] = max(m[0], key[q]);
    }
  }
};

template <int CL>
constexpr int kManyThreads = CL > 16 ? 512 : 640;

template <typename X, int CL, bool GROUPED>
__global__ void __launch_bounds__(kManyThreads<CL>, 1) score_many_kernel(const __grid_constant__ ScoreArgs a) {
  constexpr bool kLossless = sizeof(X) == 2;            // a bf16 logit is all leading bits:
  constexpr uint32_t kIndex = (kLossless ? 8 : 1) * CL - 1;    // a key then holds the expert's index, else that in the lane
  constexpr float kLead = (kIndex + 1) * 0x1p-23f;      // what it takes from the value, relative to it
  constexpr int V = CL * (int)sizeof(X) < 16 ? CL : 16 / (int)sizeof(X);
  __shared__ int hist[8 * CL];
  __shared__ __align__(16) float bias[8 * (CL + 4)];    // (rows of lanes apart by 4 banks)
  __shared__ uint2 slots[kManyThreads<CL> / 32][33];
  __shared__ int units;
  let_next_start();
  for (int e = threadIdx.x; e < 8 * CL; e += kManyThreads<CL>) hist[e] = 0;
  if (threadIdx.x == 0) units = 0;
  wait_for_previous();
  bool bad = false, unused = false;
  const bool by_logit = !a.bias && (!GROUPED || a.group_top == 1);
  for (int e = threadIdx.x; e < 8 * CL; e += kManyThreads<CL>) {
    float b = 0.f;
    if (a.bias && e < a.E) {
      b = bias_of(a, e);
      if (!(fabsf(a.bias[e]) < INFINITY)) bad = true;
    }
    bias[e / CL * (CL + 4) + e % CL] = b;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, sl = lane & 7, first = lane & 24;
  const unsigned below = ((1u << sl) - 1u) << first;
  uint2* slot = slots[threadIdx.x >> 5];
  int* slot_e = reinterpret_cast<int*>(slot);           // [4 tokens][16]
  const float* my_bias = bias + sl * (CL + 4);
  const uint32_t index0 = kIndex - (kLossless ? sl * CL : 0);   // a key's index of the lane's first expert
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
#pragma unroll
    for (int i = 0; i < CL / V; ++i) {
      const int e = sl * CL + i * V;
      uint32_t w[4] = {0, 0, 0, 0};
      if (e < a.E) {
        if constexpr (V * sizeof(X) == 16) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + e));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(row + e));
          w[0] = x.x; w[1] = x.y;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
        u[i * V + j] = sizeof(X) == 4 ? __uint_as_float(w[j & 3]) : j & 1 ? bf16_hi(w[(j / 2) & 3]) : bf16_lo(w[(j / 2) & 3]);
    }
#pragma unroll
    for (int q = 0; q < CL; q += 2)                     // NaN after an infinity or a NaN
      finite = rows::fma2(rows::f2(u[q], u[q + 1]), rows::f2(0.f, 0.f), finite);
    const bool plain = !__any_sync(kAll, rows::sum2(finite) != 0.f) && a.E == 8 * CL;
    if (!plain) {
#pragma unroll
      for (int q = 0; q < CL; ++q) {
        const bool there = sl * CL + q < a.E;
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
    // the keys; what is no expert counts as a masked one behind them
    uint32_t key[CL];
    BestKeys<CL> best;
    best.clear();
    auto take = [&](int q, float v) {
      key[q] = (key_of(v) & ~kIndex) | (index0 - q);
      best.insert(key[q]);
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
      uint32_t g1 = best.m[0], g2 = best.m[1];
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
        if (a.seg == 1 && a.sigmoid && !by_logit && __any_sync(kAll, again)) {
          // a lane's own best, if no third one comes near the last of them
          const float last = leading(a.group_top == 1 ? best.m[0] : best.m[1]);
          const float next = leading(a.group_top == 1 ? best.m[1] : best.m[2]);
          const bool live = own < a.groups && last > -INFINITY;
          bool unsure = live && next > -INFINITY && !(last - next > near_of<CL>(a.sigmoid, inv, last) + kLead * fabsf(last));
          const int q0 = (index0 - (best.m[0] & kIndex)) & (CL - 1), q1 = (index0 - (best.m[1] & kIndex)) & (CL - 1);
          const bool two = live && a.group_top == 2;
          const bool s = better_groups(a, live ? logit(a, row, sl * CL + q0, &unused) : 0.f, live ? my_bias[q0] : 0.f,
                                       two ? logit(a, row, sl * CL + q1, &unused) : 0.f, two ? my_bias[q1] : 0.f, live, own,
                                       first, 0, top, Pair{}, &unsure);
          const unsigned open = __ballot_sync(kAll, unsure);
          if (again && !(open >> first & 0xffu)) {
            stays = s;
            again = false;
          }
        }
      }
      if (!stays) best.clear();
    }
    // rounds of a maximum over the token's lanes: k, and more while the next may be as good as the k-th
    uint32_t sel = 0;
    int n = 0;
    float last = -INFINITY;
    bool stop = false;
    for (int i = 0; i < 16; ++i) {
      const uint32_t m = max8(best.m[0]);
      if (i >= a.k) {
        const float v = leading(m);
        const float gap = by_logit ? 0.f : near_of<CL>(a.sigmoid, inv, fmaxf(fabsf(last), fabsf(v))) + kLead * fabsf(v);
        stop = stop || (by_logit && kLossless) || !(v > -INFINITY) || last - v > gap;
        if (!__any_sync(kAll, !stop)) break;
      } else if (i == a.k - 1) {
        last = leading(m);
      }
      const unsigned who = __ballot_sync(kAll, best.m[0] == m);
      if (!stop) {
        ++n;
        if (sl == i) sel = m;
        if (best.m[0] == m && !(who & below)) {         // (of equal ones the first lane)
          slot_e[first * 2 + i] = (kLossless ? 0 : sl * CL) + (int)(kIndex - (m & kIndex));
          best.pop(key);
        }
      }
    }
    __syncwarp();
    int e = sl < n ? slot_e[first * 2 + sl] : 0;
    float l = sl < n ? logit(a, row, e, &unused) : -INFINITY;
    if (!(by_logit && kLossless)) {
      // (equal keys of two lanes came by their place in the lane: masked ones are chosen again)
      if (!kLossless && !(last > -INFINITY)) again = true;
      // is the order of neighbours certain?
      const float v = leading(sel), pv = __shfl_up_sync(kAll, v, 1, 8), pl = __shfl_up_sync(kAll, l, 1, 8);
      const float b = sl < n ? bias[e / CL * (CL + 4) + e % CL] : 0.f, pb = __shfl_up_sync(kAll, b, 1, 8);
      const float gap = by_logit ? 0.f : near_of<CL>(a.sigmoid, inv, fmaxf(fabsf(pv), fabsf(v))) + kLead * fabsf(v);
      const int pe = __shfl_up_sync(kAll, e, 1, 8);
      const bool close = sl > 0 && v > -INFINITY && !(pv - v > gap) && !(pl == l && pb == b && pe < e);
      bool open = again || n == 16;              // (16: there may be more)
      if (__any_sync(kAll, close || n > a.k || open)) {
        const int e2 = sl + 8 < n ? slot_e[first * 2 + sl + 8] : 0;
        const float l2 = sl + 8 < n ? logit(a, row, e2, &unused) : -INFINITY;
        const float b2 = sl + 8 < n ? bias[e2 / CL * (CL + 4) + e2 % CL] : 0.f;
        e = order8<X, CL>(a, row, e, e2, l, l2, b, b2, n, top, inv, slot_e);
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
      const bool small = !(__ballot_sync(kAll, l > -60.f) >> first & 0xffu);
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
  for (int e = threadIdx.x; e < a.E; e += kManyThreads<CL>) a.hist[(int64_t)blockIdx.x * padded4(a.E) + e] = hist[e];
}

// ---------------------------------------------------------- permutation
// Blocks [0, nb): rows of this block's assignments.  Every block adds the
// router's histograms up by itself (their sum over all blocks gives the rows'
// start of each expert, that over the blocks before it its own share), which
// saves a launch between the two.  Blocks from nb on: the rows without an assignment.
__global__ void __launch_bounds__(1024) place_kernel(const __grid_constant__ PlaceArgs a) {
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
#pragma unroll 10
    for (int i = slice; i < a.nb; i += slices) {
      const int4 c = *reinterpret_cast<const int4*>(a.hist + (int64_t)i * padded4(a.E) + e4);
      total.x += c.x; total.y += c.y; total.z += c.z; total.w += c.w;
      if (i < b) {
        before.x += c.x; before.y += c.y; before.z += c.z; before.w += c.w;
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
  scan_experts(cnt, a.E, off, start, scan);
  if (b == 0)
    for (int i = threadIdx.x; i <= a.E; i += blockDim.x) {
      if (i < a.E) a.counts[i] = cnt[i];
      a.offsets[i] = off[i];
      a.padded[i] = start[i];
    }
  if (b >= a.nb) {
    fill_rows(a, cnt, start, a.max_rows, b - a.nb, gridDim.x - a.nb);
    return;
  }
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) run[i] += start[i];
  __syncthreads();
  const int64_t t0 = (int64_t)b * a.per_block;
  place_tokens(a, t0, min((int64_t)a.T, t0 + a.per_block), run, dyn);
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
// kFusedTokens.
constexpr int kMostBlocks = 152, kFusedTokens = 32;
int tokens_per_block(int T) {
  const int per = (int)(((int64_t)T + kMostBlocks - 1) / kMostBlocks);
  return T <= kFusedTokens ? kFusedTokens : per < 4 ? 4 : per;
}

// Words of 32 tokens that a round of the placement takes: what a block has, up to
// 28 KB of bits.
int place_words(int per_block, int E) {
  const int need = (per_block + 31) / 32, most = 7168 / E;
  return need < most ? need : most;
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
    const int smem = ((3 + p.words) * a.E + 2) * 4;
    return launch_overlapped(score_route_kernel<X, C, GROUPED, true>, 1 + (unsigned)((p.max_rows - p.sure) / 4096),
                             threads, smem, s, a, p);
  }
  const int threads = 32 * warps > most ? most : 32 * warps;
  return launch_overlapped(score_route_kernel<X, C, GROUPED, false>, blocks, threads, 0, s, a, p);
}
template <typename X, int C>
cudaError_t run_score(const ScoreArgs& a, const PlaceArgs& p, int blocks, cudaStream_t s) {
  return a.groups > 1 ? run_score<X, C, true>(a, p, blocks, s) : run_score<X, C, false>(a, p, blocks, s);
}
// Eight lanes per token: for at least kManyTokens per block (the same work with a
// longer way through it: XX).
constexpr int kManyTokens = 32;
template <typename X, int CL>
cudaError_t run_many(ScoreArgs a, int blocks, bool* taken, cudaStream_t s) {
  constexpr int kVec = CL * (int)sizeof(X) < 16 ? CL * (int)sizeof(X) : 16;
  a.seg = a.group_size % CL ? 0 : a.group_size / CL;
  for (a.seg_log = 0; 1 << a.seg_log < a.seg;) ++a.seg_log;
  *taken = ((uintptr_t)a.logits & (kVec - 1)) == 0 && a.ld * sizeof(X) % kVec == 0 && a.E * sizeof(X) % kVec == 0 &&
           (a.groups == 1 || (a.seg > 0 && !(a.seg & (a.seg - 1))));
  if (!*taken) return cudaSuccess;
  return a.groups > 1 ? launch_overlapped(score_many_kernel<X, CL, true>, blocks, kManyThreads<CL>, 0, s, a)
                      : launch_overlapped(score_many_kernel<X, CL, false>, blocks, kManyThreads<CL>, 0, s, a);
}

template <typename X>
cudaError_t run_score(const ScoreArgs& a, const PlaceArgs& p, int blocks, cudaStream_t s) {
  if (a.per_block >= kManyTokens && blocks > 1 && a.k <= 8 && a.E <= 256) {
    bool taken = false;
    const cudaError_t e = a.E <= 32 ? run_many<X, 4>(a, blocks, &taken, s)
                          : a.E <= 64 ? run_many<X, 8>(a, blocks, &taken, s)
                          : a.E <= 128 ? run_many<X, 16>(a, blocks, &taken, s)
                                       : run_many<X, 32>(a, blocks, &taken, s);
    if (e != cudaSuccess || taken) return e;
  }
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
  return 16 + nb * padded4(d.E) * sizeof(int32_t);
}

cudaError_t launch_router(const moe_router_dims& d, const void* logits, const float* bias, const moe_route_out& o,
                          int32_t* hist, int32_t* status, cudaStream_t s) {
  const int per = tokens_per_block(d.T);
  const int nb = (int)(((int64_t)d.T + per - 1) / per);
  const int64_t max_rows = (int64_t)d.T * d.top_k + (int64_t)kAlign * d.E;
  const int words = place_words(per, d.E);
  const int64_t n = (int64_t)d.T * d.top_k, sure = n + (kAlign - 1) * (n < d.E ? n : d.E);
  const PlaceArgs p{o.topk_idx, hist, d.T, d.top_k, d.E, nb, per, words, max_rows, sure, o.counts, o.offsets,
                    o.padded_offsets, o.row_of_assign, o.assign_of_row};
  if (nb > 0) {
    const ScoreArgs a{logits, bias, d.ld, d.T, d.E, d.top_k, per, d.groups, d.E / d.groups, d.top_groups,
                      d.group_top, 0, 0, d.score == MOE_SCORE_SIGMOID, d.renormalise != 0, 0, d.scale, o.topk_idx,
                      o.gate, hist, status};
    const cudaError_t e = d.type == MOE_TYPE_BF16 ? run_score<__nv_bfloat16>(a, p, nb, s) : run_score<float>(a, p, nb, s);
    if (e != cudaSuccess || nb == 1) return e;
  }
  const int64_t fill = ((int64_t)kAlign * d.E + 8191) / 8192;
  return launch_overlapped(place_kernel, nb + (unsigned)fill, 1024, words * d.E * 4, s, p);
}

cudaError_t launch_router_backward(const moe_router_dims& d, const moe_route_out& o, const void* logits,
                                   const float* dgate, void* dlogits, int32_t* status, cudaStream_t s) {
  if (d.T == 0) return cudaSuccess;
  const int vec = ((uintptr_t)dlogits & 15) == 0 && d.E * (d.type == MOE_TYPE_BF16 ? 2 : 4) % 16 == 0;
  const ScoreBwdArgs a{logits, o.topk_idx, o.gate, dgate, dlogits, d.ld, d.T, d.E, d.top_k,
                       d.score == MOE_SCORE_SIGMOID, d.renormalise != 0, vec, d.scale, status};
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
