// Device helpers of the row kernels (RMS norm, activation) on either side of
// the a8w8 GEMM, gfx950: 16-byte vectors of a row through range-checked buffer
// operations, sums and maxima over a row's wavefronts, per-token and block-wise
// casts of float32 values, and the activation functions.
#pragma once

#include "hq_device.h"

namespace hq {

typedef float row_f2 __attribute__((ext_vector_type(2)));
typedef __bf16 row_b2 __attribute__((ext_vector_type(2)));

// ---- range-checked row access ---------------------------------------------------
// A row (or part of one) as a raw buffer resource: base and extent sit in scalar
// registers, loads at or past the extent read zero and stores there are dropped,
// so a row's tail needs no branch. `rows_left` <= 0 gives an empty extent.
constexpr int kRowRsrcFlags = 0x00020000;  // raw buffer, 32-bit format, range-checked
constexpr int kStreamPolicy = 2;           // non-temporal: written or read once

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, kRowRsrcFlags);
}
__device__ __forceinline__ uint4 row_load16(__amdgpu_buffer_rsrc_t r, int off) {
  const hq_u4v v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
template <int AUX>
__device__ __forceinline__ void row_store16(__amdgpu_buffer_rsrc_t r, int off, const uint4& v) {
  __builtin_amdgcn_raw_buffer_store_b128(hq_u4v{v.x, v.y, v.z, v.w}, r, off, 0, AUX);
}
// E codes (E / 4 words).
template <int E, int AUX>
__device__ __forceinline__ void row_store_codes(__amdgpu_buffer_rsrc_t r, int off, const uint32_t* w) {
  if constexpr (E == 8) __builtin_amdgcn_raw_buffer_store_b64(hq_u2v{w[0], w[1]}, r, off, 0, AUX);
  else __builtin_amdgcn_raw_buffer_store_b32(w[0], r, off, 0, AUX);
}
template <int E>
__device__ __forceinline__ void row_load_codes(__amdgpu_buffer_rsrc_t r, int off, uint32_t* w) {
  if constexpr (E == 8) {
    const hq_u2v v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
    w[0] = v[0];
    w[1] = v[1];
  } else {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
}

// A vector's elements as float32, and float32 values as a vector of the type
// (bf16: round to nearest even, two per v_cvt_pk_bf16_f32).
template <int XT>
__device__ __forceinline__ void vec_widen(const uint4& v, float* f) {
#pragma unroll
  for (int e = 0; e < VecTraits<XT>::kElems; ++e) f[e] = vec_elem<XT>(v, e);
}
template <int XT>
__device__ __forceinline__ uint4 vec_narrow(const float* f) {
  if constexpr (XT == kF32) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((row_f2{f[2 * i], f[2 * i + 1]}), row_b2));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---- reductions -----------------------------------------------------------------
// Sum over the 64 lanes, returned to every lane, in one fixed order. The lane
// moves are those of wave_max_u32; rows outside a broadcast's row mask add 0.
__device__ __forceinline__ float wave_sum_f32(float v) {
#define HQ_DPP_ADD(CTRL, MASK) \
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, MASK, 0xF, false))
  HQ_DPP_ADD(0xB1, 0xF);   // swap neighbours
  HQ_DPP_ADD(0x4E, 0xF);   // swap pairs
  HQ_DPP_ADD(0x141, 0xF);  // half-row mirror
  HQ_DPP_ADD(0x140, 0xF);  // row mirror
  HQ_DPP_ADD(0x142, 0xA);  // lane 15 of rows 0 and 2 to rows 1 and 3
  HQ_DPP_ADD(0x143, 0xC);  // lane 31 to rows 2 and 3
#undef HQ_DPP_ADD
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Max over aligned groups of g lanes (g = 4, 8, 16 or 32, wavefront-uniform);
// every lane of a group gets its group's max.
__device__ __forceinline__ uint32_t lanes_max_u32(uint32_t v, int g) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  if (g >= 8) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  if (g >= 16) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  if (g >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
  return v;
}

// A row's total from its WPR wavefronts' partials. `slot` has one entry per
// wavefront of the row and is not written again before the next barrier that
// follows the reads. WPR == 1 needs no barrier; otherwise every wavefront of
// the workgroup calls this.
template <int WPR>
__device__ __forceinline__ float row_sum_f32(float v, float* slot, int wave) {
  v = wave_sum_f32(v);
  if constexpr (WPR == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[wave] = v;
  __syncthreads();
  float t = slot[0];
#pragma unroll
  for (int i = 1; i < WPR; ++i) t += slot[i];
  return t;
}
// Two totals in one exchange.
template <int WPR>
__device__ __forceinline__ void row_sum2_f32(float v, float u, float* slot, float* slot2, int wave, float* vs, float* us) {
  v = wave_sum_f32(v);
  u = wave_sum_f32(u);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) {
      slot[wave] = v;
      slot2[wave] = u;
    }
    __syncthreads();
    v = slot[0];
    u = slot2[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      v += slot[i];
      u += slot2[i];
    }
  }
  *vs = v;
  *us = u;
}
template <int WPR>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v, uint32_t* slot, int wave) {
  v = wave_max_u32(v);
  if constexpr (WPR == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[wave] = v;
  __syncthreads();
  uint32_t t = slot[0];
#pragma unroll
  for (int i = 1; i < WPR; ++i) t = max(t, slot[i]);
  return t;
}

// ---- casts of float32 values ------------------------------------------------------
// Largest magnitude of n values as float32 bits, Inf and NaN included; and over
// the finite ones only.
template <int N>
__device__ __forceinline__ uint32_t absmax_raw(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  return m;
}
template <int N>
__device__ __forceinline__ uint32_t absmax_finite(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const uint32_t a = __float_as_uint(v[e]) & 0x7fffffffu;
    m = max(m, a < kInfBits ? a : 0u);
  }
  return m;
}

// N codes of fl32(v * r). `special`: some value is Inf or NaN (clamp and NaN
// patch). Otherwise r comes from the amax of the values' own group, so no
// scaled value passes fmax by more than one ulp (see cvt2).
template <int FMT, int N>
__device__ __forceinline__ void cast_values(const float* v, float r, bool special, uint32_t* w) {
#pragma unroll
  for (int d = 0; d < N / 4; ++d) {
    const float a = v[4 * d] * r, b = v[4 * d + 1] * r, c = v[4 * d + 2] * r, e = v[4 * d + 3] * r;
    w[d] = special ? patch_nan4(cvt4<FMT, true>(a, b, c, e), a, b, c, e) : cvt4<FMT, false>(a, b, c, e);
  }
}

// One vector of an E4M3 block-wise checkpoint: E values per lane, a block is
// the g = block_size / E lanes from a multiple of g on. Codes and the block's
// scale, which is lane-uniform within the block.
template <int E>
__device__ __forceinline__ float checkpoint_vec(const float* v, int g, uint32_t* w) {
  const uint32_t raw = absmax_raw<E>(v);
  uint32_t fin = raw;
  const bool special = __any(raw >= kInfBits);  // rare, wavefront-uniform
  if (special) fin = absmax_finite<E>(v);
  const float s = scale_from_amax<kE4M3>(__uint_as_float(lanes_max_u32(fin, g)));
  cast_values<kE4M3, E>(v, 1.0f / s, special, w);
  return s;
}

// E codes decoded and scaled (E4M3).
template <int E>
__device__ __forceinline__ void decode_vec(const uint32_t* w, float s, float* f) {
#pragma unroll
  for (int d = 0; d < E / 4; ++d) {
    const row_f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[d], false);
    const row_f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[d], true);
    f[4 * d] = lo[0] * s;
    f[4 * d + 1] = lo[1] * s;
    f[4 * d + 2] = hi[0] * s;
    f[4 * d + 3] = hi[1] * s;
  }
}

// ---- sums over rows in one workgroup ---------------------------------------------
// A workgroup of 1024 threads holds 8 vector columns (128 bytes of a row) of 128
// rows at a time: lane l of wavefront w is column l % 8 of row slot 8 w + l / 8.
// N values per thread are added over the slots in a fixed order; threads 0 .. 7
// return true with their column's sums in v. `s` holds 16 * 8 * N floats.
constexpr int kColVecs = 8, kColSlots = 128;
template <int N>
__device__ __forceinline__ bool slots_sum(float* v, float* s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    v[e] += __shfl_xor(v[e], 8, 64);
    v[e] += __shfl_xor(v[e], 16, 64);
    v[e] += __shfl_xor(v[e], 32, 64);
  }
  if (lane < 8) {
#pragma unroll
    for (int e = 0; e < N; ++e) s[(wave * N + e) * 8 + lane] = v[e];
  }
  __syncthreads();
  if (threadIdx.x >= 8) return false;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    v[e] = s[e * 8 + lane];
#pragma unroll
    for (int w = 1; w < 16; ++w) v[e] += s[(w * N + e) * 8 + lane];
  }
  return true;
}

}  // namespace hq
