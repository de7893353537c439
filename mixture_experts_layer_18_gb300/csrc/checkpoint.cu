// checkpoint.cu - the layer's activations kept as MXFP8 between its forward and
// its backward, and the decoding of MXFP8 rows.
//
// Between the two passes of a layer the backward needs X_perm, h13 and act
// (moe_saved_layout): X_perm is X gathered, act follows from h13 and the gates, so
// X [T, H] and h13 in the order of the assignments [T k, 2I] hold all of it, and as
// E4M3 codes with a scale per 32 columns (the rule of quant.cu) they take
// 33/32 bytes per element.
//   save      codes of X[t], and of h13[row_of_assign[a]] for every assignment a
//   restore   X_perm[r] = X~[a / k], h13[r] = h~[a], act[r] = silu(u~) v~ (times the
//             gate where `act` holds gate * A), r = row_of_assign[a]; pad rows 0
// (~: decoded).  Both are bound by HBM: a warp takes a piece of a row at a time,
// 8 neighbouring columns per lane, four lanes to a block of 32.  A token's codes
// are decoded once and stored to its k rows.
//
// Measured (GB300, 16384 tokens, 8 of 128 experts, bf16): H 2048, I 768 save 117 us (6.1
// TB/s), restore 220 us (6.5 TB/s); H 4096, I 1536 207 us (6.9) and 441 us (6.6).
#include "mx_encode.cuh"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ int64_t grid_warps() { return ((int64_t)gridDim.x * blockDim.x) >> 5; }
__device__ __forceinline__ int64_t global_warp() {
  return ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
}

// 8 neighbouring elements (p on a 16-byte boundary).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) { rows::load_part(p, v); }
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) { rows::store_part(p, v); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Codes of a lane's 8 columns; the four lanes of a block join its maximum.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], int* scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
  top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
  top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
  *scale = mx_scale_byte(top);
  const float inv = mx_inv_scale(*scale);
  return make_uint2(e4m3x2(v[0] * inv, v[1] * inv) | (uint32_t)e4m3x2(v[2] * inv, v[3] * inv) << 16,
                    e4m3x2(v[4] * inv, v[5] * inv) | (uint32_t)e4m3x2(v[6] * inv, v[7] * inv) << 16);
}

// The values of 8 codes under one scale (exact in fp32).
__device__ __forceinline__ void decode8(uint2 q, int scale, float (&v)[8]) {
  const float s = __uint_as_float(scale ? (uint32_t)scale << 23 : 1u << 22);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (i < 2 ? q.x : q.y) >> (16 * (i & 1));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

struct CkptArgs {
  const void* X;            // save; null: its codes are there already
  void* x_perm;             // restore
  void* h13;
  void* act;
  uint8_t* x_q;
  uint8_t* x_s;
  uint8_t* h_q;
  uint8_t* h_s;
  const float* gate;        // restore, null where `act` is not gated
  const int32_t* row_of_assign;
  const int32_t* padded_offsets;
  const int32_t* counts;
  int64_t n_assign;
  int T, H, I, E, k;
  int32_t* status;
};

// Steps of 256 columns in a warp's unit of work: of a row to save or to decode; of
// a token's row to restore (stored k times); of each half of h13 to restore.
// (16384 tokens, 8 of 128, H 2048.  Save: I 768 117 us with 4, 137 with 2, 141 with 8; I 512 77,
// 99, 124; I 1024 136, 178, 171.  Restore with 2 steps of X and 3 of a half: I 768 220 us, I 512
// 184, I 1024 276, I 1408 329; with 2 and 4 220, 182, 261, 329; 2 and 2 223, 178, 263, 330; 4
// and 3 241, 209, 319, 371; 1 and 3 222, 181, 268, 329.)
constexpr int kPieces = 4, kTokenPieces = 2, kHalfPieces = 3;
constexpr int kUnit = 256 * kPieces;

// A row's codes of the columns [c0, c0 + kUnit).
template <typename X>
__device__ __forceinline__ void save_unit(const X* src, uint8_t* q, uint8_t* s, int c0, int C, int lane) {
  float v[kPieces][8];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = c0 + i * 256 + lane * 8;
    if (c < C) {
      load8(src + c, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = c0 + i * 256 + lane * 8;
    int sb;
    const uint2 w = encode8(v[i], &sb);
    if (c < C) {
      *reinterpret_cast<uint2*>(q + c) = w;
      if ((lane & 3) == 0) s[c >> 5] = (uint8_t)sb;
    }
  }
}

template <typename X>
__global__ void __launch_bounds__(kThreads) ckpt_save_kernel(const __grid_constant__ CkptArgs a) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int rows = (int)min((int64_t)a.padded_offsets[a.E], a.n_assign + (int64_t)kAlign * a.E);
  const int nx = (a.H + kUnit - 1) / kUnit, nh = (2 * a.I + kUnit - 1) / kUnit;
  const int64_t ux = a.X ? (int64_t)a.T * nx : 0, all = ux + a.n_assign * nh;
  for (int64_t u = global_warp(); u < all; u += grid_warps()) {
    if (u < ux) {
      const int64_t t = u / nx;
      save_unit(static_cast<const X*>(a.X) + t * a.H, a.x_q + t * a.H, a.x_s + t * (a.H >> 5),
                (int)(u - t * nx) * kUnit, a.H, lane);
    } else {
      const int64_t n = (u - ux) / nh;
      const int r = a.row_of_assign[n], C = 2 * a.I;
      if (r < 0 || r >= rows) {
        if (lane == 0) report(a.status, MOE_ERR_BAD_INDEX);
        continue;
      }
      save_unit(static_cast<const X*>(a.h13) + (int64_t)r * C, a.h_q + n * C, a.h_s + n * (C >> 5),
                (int)(u - ux - n * nh) * kUnit, C, lane);
    }
  }
}

template <typename X>
__device__ __forceinline__ void zero_row(X* p, int C, int lane) {
  const float z[8] = {};
  for (int c = lane * 8; c < C; c += 256) store8(p + c, z);
}

template <typename X>
__global__ void __launch_bounds__(kThreads) ckpt_restore_kernel(const __grid_constant__ CkptArgs a) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int rows = (int)min((int64_t)a.padded_offsets[a.E], a.n_assign + (int64_t)kAlign * a.E);
  X* x_perm = static_cast<X*>(a.x_perm);
  X* h13 = static_cast<X*>(a.h13);
  X* act = static_cast<X*>(a.act);
  const int nx = (a.H + 256 * kTokenPieces - 1) / (256 * kTokenPieces);
  const int nh = (a.I + 256 * kHalfPieces - 1) / (256 * kHalfPieces);
  const int64_t up = (int64_t)a.E * kAlign, ux = up + (int64_t)a.T * nx, all = ux + a.n_assign * nh;
  for (int64_t u = global_warp(); u < all; u += grid_warps()) {
    if (u < up) {                          // the i-th row behind an expert's, as the forward leaves it
      const int e = (int)(u / kAlign);
      const int64_t r = (int64_t)a.padded_offsets[e] + a.counts[e] + u % kAlign;
      if (r >= a.padded_offsets[e + 1] || r < 0 || r >= rows) continue;
      zero_row(x_perm + r * a.H, a.H, lane);
      zero_row(h13 + r * 2 * a.I, 2 * a.I, lane);
      zero_row(act + r * a.I, a.I, lane);
      continue;
    }
    if (u < ux) {
      const int64_t t = (u - up) / nx;
      const int c0 = (int)(u - up - t * nx) * (256 * kTokenPieces);
      int my = -1;                         // lane j < k: the row of slot j
      if (lane < a.k) {
        my = a.row_of_assign[t * a.k + lane];
        if (my < 0 || my >= rows) {
          report(a.status, MOE_ERR_BAD_INDEX);
          my = -1;
        }
      }
      uint2 q[kTokenPieces];
      int s[kTokenPieces];
#pragma unroll
      for (int i = 0; i < kTokenPieces; ++i) {
        const int c = c0 + i * 256 + lane * 8;
        if (c < a.H) {
          q[i] = *reinterpret_cast<const uint2*>(a.x_q + t * a.H + c);
          s[i] = a.x_s[t * (a.H >> 5) + (c >> 5)];
        }
      }
      float v[kTokenPieces][8];
#pragma unroll
      for (int i = 0; i < kTokenPieces; ++i) decode8(q[i], s[i], v[i]);
      for (int j = 0; j < a.k; ++j) {
        const int r = __shfl_sync(kAll, my, j);
        if (r < 0) continue;
        X* d = x_perm + (int64_t)r * a.H;
#pragma unroll
        for (int i = 0; i < kTokenPieces; ++i) {
          const int c = c0 + i * 256 + lane * 8;
          if (c < a.H) store8(d + c, v[i]);
        }
      }
      continue;
    }
    const int64_t n = (u - ux) / nh;
    const int r = a.row_of_assign[n];
    if (r < 0 || r >= rows) {
      if (lane == 0) report(a.status, MOE_ERR_BAD_INDEX);
      continue;
    }
    const int c0 = (int)(u - ux - n * nh) * (256 * kHalfPieces);
    const float g = a.gate ? a.gate[n] : 1.f;
    const uint8_t* hq = a.h_q + n * 2 * a.I;
    const uint8_t* hs = a.h_s + n * (2 * a.I >> 5);
    uint2 q[kHalfPieces][2];
    int s[kHalfPieces][2];
#pragma unroll
    for (int i = 0; i < kHalfPieces; ++i) {
      const int c = c0 + i * 256 + lane * 8;
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (c < a.I) {
          q[i][p] = *reinterpret_cast<const uint2*>(hq + p * a.I + c);
          s[i][p] = hs[(p * a.I + c) >> 5];
        }
    }
#pragma unroll
    for (int i = 0; i < kHalfPieces; ++i) {
      const int c = c0 + i * 256 + lane * 8;
      if (c >= a.I) continue;
      float x[8], v[8];
      decode8(q[i][0], s[i][0], x);
      decode8(q[i][1], s[i][1], v);
      X* h = h13 + (int64_t)r * 2 * a.I + c;
      store8(h, x);
      store8(h + a.I, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fdividef(x[e], 1.f + __expf(-x[e])) * v[e] * g;
      store8(act + (int64_t)r * a.I + c, x);
    }
  }
}

// Rows of codes back to numbers; VEC: rows of dst start on 16-byte boundaries.
template <typename X, bool VEC>
__global__ void __launch_bounds__(kThreads) decode_kernel(const uint8_t* q, const uint8_t* s, int R, int C, int64_t ld,
                                                          X* dst) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int nu = (C + kUnit - 1) / kUnit;
  const int64_t all = (int64_t)R * nu;
  for (int64_t u = global_warp(); u < all; u += grid_warps()) {
    const int64_t r = u / nu;
    const int c0 = (int)(u - r * nu) * kUnit;
    uint2 w[kPieces];
    int sb[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = c0 + i * 256 + lane * 8;
      if (c < C) {
        w[i] = *reinterpret_cast<const uint2*>(q + r * C + c);
        sb[i] = s[r * (C >> 5) + (c >> 5)];
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = c0 + i * 256 + lane * 8;
      if (c >= C) continue;
      float v[8];
      decode8(w[i], sb[i], v);
      X* d = dst + r * ld + c;
      if constexpr (VEC) {
        store8(d, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) rows::put(d + e, v[e]);
      }
    }
  }
}

// Blocks for `units` warps' worth of work: at most `per_sm` per SM.  (Saving reads
// most: eight, all there is room for; writing more it goes faster with blocks that come
// and go: restoring as above 457 us with eight and H 4096, I 1536, 440 with 64; H 2048, I 768
// 230 and 220.)
unsigned blocks_for(int64_t units, int per_sm) {
  const int64_t need = (units + kThreads / 32 - 1) / (kThreads / 32), most = (int64_t)sm_count() * per_sm;
  return (unsigned)(need < 1 ? 1 : need < most ? need : most);
}

CkptArgs ckpt_args(const CheckpointDesc& d) {
  return CkptArgs{d.X, d.x_perm, d.h13, d.act, d.x_q, d.x_s, d.h_q, d.h_s, d.gate, d.row_of_assign, d.padded_offsets,
                  d.counts, (int64_t)d.T * d.k, d.T, d.H, d.I, d.E, d.k, d.status};
}

}  // namespace

cudaError_t launch_checkpoint_save(const CheckpointDesc& d, cudaStream_t s) {
  if (d.T == 0) return cudaSuccess;
  const CkptArgs a = ckpt_args(d);
  const int64_t units = (d.X ? (int64_t)d.T * ((d.H + kUnit - 1) / kUnit) : 0) +
                        a.n_assign * ((2 * d.I + kUnit - 1) / kUnit);
  const unsigned grid = blocks_for(units, 8);
  return d.elem_bytes == 2 ? launch_overlapped(ckpt_save_kernel<__nv_bfloat16>, grid, kThreads, 0, s, a)
                           : launch_overlapped(ckpt_save_kernel<float>, grid, kThreads, 0, s, a);
}

cudaError_t launch_checkpoint_restore(const CheckpointDesc& d, cudaStream_t s) {
  if (d.T == 0) return cudaSuccess;
  const CkptArgs a = ckpt_args(d);
  const int64_t units = (int64_t)d.E * kAlign +
                        (int64_t)d.T * ((d.H + 256 * kTokenPieces - 1) / (256 * kTokenPieces)) +
                        a.n_assign * ((d.I + 256 * kHalfPieces - 1) / (256 * kHalfPieces));
  const unsigned grid = blocks_for(units, 64);
  return d.elem_bytes == 2 ? launch_overlapped(ckpt_restore_kernel<__nv_bfloat16>, grid, kThreads, 0, s, a)
                           : launch_overlapped(ckpt_restore_kernel<float>, grid, kThreads, 0, s, a);
}

cudaError_t launch_dequantize(const uint8_t* q, const uint8_t* sf, int R, int C, int64_t ld, int type, void* dst,
                              cudaStream_t s) {
  if (R == 0) return cudaSuccess;
  const unsigned grid = blocks_for((int64_t)R * ((C + kUnit - 1) / kUnit), 64);
  const int es = type == MOE_TYPE_BF16 ? 2 : 4;
  const bool vec = ((uintptr_t)dst & 15) == 0 && (R == 1 || ld * es % 16 == 0);
  if (es == 2)
    return vec ? launch_overlapped(decode_kernel<__nv_bfloat16, true>, grid, kThreads, 0, s, q, sf, R, C, ld,
                                   static_cast<__nv_bfloat16*>(dst))
               : launch_overlapped(decode_kernel<__nv_bfloat16, false>, grid, kThreads, 0, s, q, sf, R, C, ld,
                                   static_cast<__nv_bfloat16*>(dst));
  return vec ? launch_overlapped(decode_kernel<float, true>, grid, kThreads, 0, s, q, sf, R, C, ld,
                                 static_cast<float*>(dst))
             : launch_overlapped(decode_kernel<float, false>, grid, kThreads, 0, s, q, sf, R, C, ld,
                                 static_cast<float*>(dst));
}

}  // namespace moe
