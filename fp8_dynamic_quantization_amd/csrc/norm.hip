// RMS norm with the residual's addition and FP8 output, and its backward pass,
// gfx950.
//
//   forward   h = x + residual            rstd = 1 / sqrt(mean_c h^2 + eps)
//             y = (h * rstd) * w          s = max(amax_row(y) / fmax, 2^-126)
//             q = cast(y * (1 / s))       optionally h itself and an 8-bit block-wise checkpoint of it
//   backward  xh = h * rstd, t = dy * w   dx = dres + rstd * (t - xh * mean_c(t * xh))
//             dw = sum_rows dy * xh
//
// All sums are float32; h enters the statistics and y unrounded.
#include "hq_launch.h"
#include "hq_row.h"

namespace hq {

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Vectors t, t + 64 WPR, ... of a row belong to thread t of its WPR wavefronts;
// NV of them stay in registers, so x and the residual are read once. Lanes past
// the row's end read zeros, which add nothing to a sum or a maximum.
template <int XT, int WPR, int NV>
struct NormFwd {
  static constexpr int E = VecTraits<XT>::kElems;
  static constexpr int kRowThreads = 64 * WPR;
  static constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;  // rows per workgroup
  static constexpr int kThreads = kRowThreads * kRows;
};

template <int XT, int WPR, int NV>
__global__ __launch_bounds__((NormFwd<XT, WPR, NV>::kThreads)) void rmsnorm_quant_kernel(NormArgs a) {
  using C = NormFwd<XT, WPR, NV>;
  constexpr int E = C::E;
  static_assert(WPR == 1 || C::kRows == 1, "one row per workgroup where a row needs its barrier");
  __shared__ float s_sum[WPR];
  __shared__ uint32_t s_max[WPR], s_fin[WPR];
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % WPR);
  const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x / C::kRowThreads);
  const int t = threadIdx.x % C::kRowThreads;
  const uint32_t row_bytes = (uint32_t)a.cols * (16 / E);
  const int off0 = t * 16;             // byte offset of vector 0 in a row; a step adds 16 kRowThreads
  const int nb = a.cblock ? (a.cols + a.cblock - 1) / a.cblock : 0;
  const int g = a.cblock / E;
  const float inv_n = 1.0f / (float)a.cols;

  uint4 w[NV];
  const __amdgpu_buffer_rsrc_t w_rsrc = row_rsrc(a.weight, a.weight ? row_bytes : 0u);
#pragma unroll
  for (int j = 0; j < NV; ++j) w[j] = row_load16(w_rsrc, off0 + j * 16 * C::kRowThreads);

  const int64_t step = (int64_t)gridDim.x * C::kRows;
  for (int64_t row = (int64_t)blockIdx.x * C::kRows + grp; row < a.rows; row += step) {
    const size_t at = (size_t)row * row_bytes;
    float v[NV][E];
    {
      const __amdgpu_buffer_rsrc_t x_rsrc = row_rsrc(static_cast<const uint8_t*>(a.x) + at, row_bytes);
      uint4 xv[NV], rv[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) xv[j] = row_load16(x_rsrc, off0 + j * 16 * C::kRowThreads);
      if (a.residual) {
        const __amdgpu_buffer_rsrc_t r_rsrc = row_rsrc(static_cast<const uint8_t*>(a.residual) + at, row_bytes);
#pragma unroll
        for (int j = 0; j < NV; ++j) rv[j] = row_load16(r_rsrc, off0 + j * 16 * C::kRowThreads);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        vec_widen<XT>(xv[j], v[j]);
        if (a.residual) {
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][e] += vec_elem<XT>(rv[j], e);
        }
      }
    }
    float ss[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      ss[j] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) ss[j] = fmaf(v[j][e], v[j][e], ss[j]);
    }
#pragma unroll
    for (int j = 1; j < NV; ++j) ss[0] += ss[j];
    if (a.h) {
      const __amdgpu_buffer_rsrc_t h_rsrc = row_rsrc(static_cast<uint8_t*>(a.h) + at, row_bytes);
#pragma unroll
      for (int j = 0; j < NV; ++j) row_store16<kStreamPolicy>(h_rsrc, off0 + j * 16 * C::kRowThreads, vec_narrow<XT>(v[j]));
    }
    if (a.cblock) {
      const __amdgpu_buffer_rsrc_t c_rsrc = row_rsrc(a.cq + (size_t)row * a.cols, (uint32_t)a.cols);
      const __amdgpu_buffer_rsrc_t cs_rsrc = row_rsrc(a.cs + (size_t)row * nb, (uint32_t)nb * 4u);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = t + j * C::kRowThreads;
        if (__builtin_amdgcn_readfirstlane(i - (int)(threadIdx.x & 63)) * E >= a.cols) break;  // wavefront past the row
        uint32_t cw[E / 4];
        const float s = checkpoint_vec<E>(v[j], g, cw);
        row_store_codes<E, kStreamPolicy>(c_rsrc, i * E, cw);
        if ((i & (g - 1)) == 0)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), cs_rsrc, i / g * 4, 0, 0);
      }
    }
    const float total = row_sum_f32<WPR>(ss[0], s_sum, wave);
    const float rstd = 1.0f / sqrtf(fmaf(total, inv_n, a.eps));
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[j][e] = a.weight ? v[j][e] * rstd * vec_elem<XT>(w[j], e) : v[j][e] * rstd;
      m = max(m, absmax_raw<E>(v[j]));
    }
    m = row_max_u32<WPR>(m, s_max, wave);
    const bool special = m >= kInfBits;  // rare, uniform over the row
    if (special) {
      m = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) m = max(m, absmax_finite<E>(v[j]));
      m = row_max_u32<WPR>(m, s_fin, wave);
    }
    const float amax = __uint_as_float(m);
    const float s = a.fmt == kE4M3 ? scale_from_amax<kE4M3>(amax) : scale_from_amax<kE5M2>(amax);
    const float r = 1.0f / s;
    const __amdgpu_buffer_rsrc_t q_rsrc = row_rsrc(a.q + (size_t)row * a.cols, (uint32_t)a.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint32_t cw[E / 4];
      if (a.fmt == kE4M3) cast_values<kE4M3, E>(v[j], r, special, cw);
      else cast_values<kE5M2, E>(v[j], r, special, cw);
      row_store_codes<E, kStreamPolicy>(q_rsrc, (t + j * C::kRowThreads) * E, cw);
    }
    if (t == 0) {
      a.scale[row] = s;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Rows longer than the register form holds: one workgroup of 16 wavefronts per
// row reads the row three times (sum of squares and checkpoint, maximum, cast
// and h). h is written in the last pass only, each vector after its own reads,
// so h may be the residual's or x's own buffer here too.
template <int XT>
__global__ __launch_bounds__(1024) void rmsnorm_quant_long_kernel(NormArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  __shared__ float s_sum[16];
  __shared__ uint32_t s_max[16], s_fin[16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = threadIdx.x;
  const int nvec = a.cols / E;
  const int nb = a.cblock ? (a.cols + a.cblock - 1) / a.cblock : 0;
  const int g = a.cblock / E;
  const float inv_n = 1.0f / (float)a.cols;
  const uint4* wv = static_cast<const uint4*>(a.weight);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint4* x = static_cast<const uint4*>(a.x) + (size_t)row * nvec;
    const uint4* res = a.residual ? static_cast<const uint4*>(a.residual) + (size_t)row * nvec : nullptr;
    auto load_h = [&](int i, float* v) {
      vec_widen<XT>(x[i], v);
      if (res) {
        const uint4 rv = res[i];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] += vec_elem<XT>(rv, e);
      }
    };
    float ss = 0.0f;
    for (int i0 = 0; i0 < nvec; i0 += 1024) {  // every lane takes part in a block's maximum
      const int i = i0 + t;
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.0f;
      if (i < nvec) load_h(i, v);
      float p = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) p = fmaf(v[e], v[e], p);
      ss += p;
      if (a.cblock) {
        uint32_t cw[E / 4];
        const float s = checkpoint_vec<E>(v, g, cw);
        if (i < nvec) {
          store_codes<E>(a.cq + (size_t)row * a.cols + (size_t)i * E, cw);
          if ((i & (g - 1)) == 0) a.cs[(size_t)row * nb + i / g] = s;
        }
      }
    }
    const float total = row_sum_f32<16>(ss, s_sum, wave);
    const float rstd = 1.0f / sqrtf(fmaf(total, inv_n, a.eps));
    auto load_y = [&](int i, float* h, float* y) {
      load_h(i, h);
      const uint4 w = wv ? wv[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = wv ? h[e] * rstd * vec_elem<XT>(w, e) : h[e] * rstd;
    };
    uint32_t raw = 0, fin = 0;
    for (int i = t; i < nvec; i += 1024) {
      float h[E], y[E];
      load_y(i, h, y);
      raw = max(raw, absmax_raw<E>(y));
      fin = max(fin, absmax_finite<E>(y));
    }
    const bool special = row_max_u32<16>(raw, s_max, wave) >= kInfBits;
    const float amax = __uint_as_float(row_max_u32<16>(fin, s_fin, wave));
    const float s = a.fmt == kE4M3 ? scale_from_amax<kE4M3>(amax) : scale_from_amax<kE5M2>(amax);
    const float r = 1.0f / s;
    for (int i = t; i < nvec; i += 1024) {
      float h[E], y[E];
      load_y(i, h, y);
      uint32_t cw[E / 4];
      if (a.fmt == kE4M3) cast_values<kE4M3, E>(y, r, special, cw);
      else cast_values<kE5M2, E>(y, r, special, cw);
      store_codes<E>(a.q + (size_t)row * a.cols + (size_t)i * E, cw);
      if (a.h) static_cast<uint4*>(a.h)[(size_t)row * nvec + i] = vec_narrow<XT>(h);
    }
    if (t == 0) {
      a.scale[row] = s;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A workgroup of 16 wavefronts holds 16 / WPR rows at a time, WPR wavefronts to
// a row, and walks down the tensor; a thread keeps its NV vectors' columns of
// dw in registers over all its rows. At the end the row groups of a workgroup
// are added in LDS in a fixed order and one partial row per workgroup goes to
// the workspace, which column_sums_kernel adds in order: dw does not depend on
// which workgroup ends first. dx goes through the caches (the next kernel reads
// it): streamed past them it took 49.3 us instead of 45.6 at 8192 x 4096 bf16 with a
// checkpoint (40.8 of it this kernel). That shape moves 236 MB, 38.4 us at 6.15 TB/s, a
// large elementwise pass's best; more workgroups per CU (51 to 63 us for 2 to 8),
// loading the next row ahead (49.5, before the stores changed) and runs of neighbouring
// rows per workgroup (49.1) were slower.
constexpr int kBwdLdsFloats = 16384;

// Few rows: dw needs nothing that dx computes (rstd is given), so the same launch
// gets workgroups of its own for it, past the `row_blocks` that compute dx. They
// read dy and h again, from the caches, and no second launch adds partial sums.
// (Where dx is dy's own buffer, they go first, in a launch of their own.)
template <int XT, bool CKPT>
__device__ __forceinline__ void rmsnorm_dw_columns(const NormBwdArgs& a, int tile, float* s) {
  constexpr int E = VecTraits<XT>::kElems;
  const int i = tile * kColVecs + (threadIdx.x & 7);  // vector column
  const int nvec = a.cols / E;
  const int nb = CKPT ? (a.cols + a.cblock - 1) / a.cblock : 0;
  const int gsh = CKPT ? __builtin_ctz(a.cblock / E) : 0;
  float dw[E];
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = 0.0f;
  if (i < nvec) {
#pragma unroll 4
    for (int row = threadIdx.x >> 3; row < a.rows; row += kColSlots) {
      const uint4 dy = static_cast<const uint4*>(a.dy)[(size_t)row * nvec + i];
      float xh[E];
      if constexpr (CKPT) {
        uint32_t w[E / 4];
        const uint32_t* p = reinterpret_cast<const uint32_t*>(a.cq + (size_t)row * a.cols + (size_t)i * E);
#pragma unroll
        for (int d = 0; d < E / 4; ++d) w[d] = p[d];
        decode_vec<E>(w, a.cs[(size_t)row * nb + (i >> gsh)], xh);
      } else {
        vec_widen<XT>(static_cast<const uint4*>(a.h)[(size_t)row * nvec + i], xh);
      }
      const float rstd = a.rstd[row];
#pragma unroll
      for (int e = 0; e < E; ++e) dw[e] = fmaf(vec_elem<XT>(dy, e), xh[e] * rstd, dw[e]);
    }
  }
  if (slots_sum<E>(dw, s) && i < nvec) {
#pragma unroll
    for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(a.dw + (size_t)i * E + e) = make_float4(dw[e], dw[e + 1], dw[e + 2], dw[e + 3]);
  }
}

template <int XT, int WPR, int NV, bool CKPT>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_kernel(NormBwdArgs a, int row_blocks) {
  constexpr int E = VecTraits<XT>::kElems;
  constexpr int kRowThreads = 64 * WPR;
  constexpr int kGroups = 16 / WPR;
  constexpr int kCols = kRowThreads * NV * E;
  static_assert(kGroups == 1 || kCols * (kGroups / 2) <= kBwdLdsFloats, "row groups meet in LDS");
  constexpr int kPart = kGroups > 1 ? kCols * (kGroups / 2) : 1;
  __shared__ float s_part[kPart < 16 * 8 * E ? 16 * 8 * E : kPart];
  __shared__ float s_sum[2][16];
  if ((int)blockIdx.x >= row_blocks) return rmsnorm_dw_columns<XT, CKPT>(a, blockIdx.x - row_blocks, s_part);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % WPR);
  const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x / kRowThreads);
  const int t = threadIdx.x % kRowThreads;
  const uint32_t row_bytes = (uint32_t)a.cols * (16 / E);
  const int off0 = t * 16;
  const int nb = CKPT ? (a.cols + a.cblock - 1) / a.cblock : 0;
  const int gsh = CKPT ? __builtin_ctz(a.cblock / E) : 0;
  const float inv_n = 1.0f / (float)a.cols;

  uint4 w[NV];
  const __amdgpu_buffer_rsrc_t w_rsrc = row_rsrc(a.weight, a.weight ? row_bytes : 0u);
#pragma unroll
  for (int j = 0; j < NV; ++j) w[j] = row_load16(w_rsrc, off0 + j * 16 * kRowThreads);
  float dw[NV][E];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[j][e] = 0.0f;

  int parity = 0;
  // the trip count is uniform over the workgroup; groups past the last row read
  // empty extents and store nothing
  for (int64_t row0 = (int64_t)blockIdx.x * kGroups; row0 < a.rows; row0 += (int64_t)row_blocks * kGroups) {
    const int64_t row = min(row0 + grp, (int64_t)a.rows - 1);
    const bool live = row0 + grp < a.rows;
    const uint32_t bytes = live ? row_bytes : 0u;
    const size_t at = (size_t)row * row_bytes;
    uint4 dy[NV], hv[NV], rv[NV];
    uint32_t hc[NV][E / 4];
    float hs[NV];
    const __amdgpu_buffer_rsrc_t y_rsrc = row_rsrc(static_cast<const uint8_t*>(a.dy) + at, bytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) dy[j] = row_load16(y_rsrc, off0 + j * 16 * kRowThreads);
    if constexpr (CKPT) {
      const __amdgpu_buffer_rsrc_t c_rsrc = row_rsrc(a.cq + (size_t)row * a.cols, live ? (uint32_t)a.cols : 0u);
      const __amdgpu_buffer_rsrc_t s_rsrc = row_rsrc(a.cs + (size_t)row * nb, live ? (uint32_t)nb * 4u : 0u);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = t + j * kRowThreads;
        row_load_codes<E>(c_rsrc, i * E, hc[j]);
        hs[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(s_rsrc, (i >> gsh) * 4, 0, 0));
      }
    } else {
      const __amdgpu_buffer_rsrc_t h_rsrc = row_rsrc(static_cast<const uint8_t*>(a.h) + at, bytes);
#pragma unroll
      for (int j = 0; j < NV; ++j) hv[j] = row_load16(h_rsrc, off0 + j * 16 * kRowThreads);
    }
    const __amdgpu_buffer_rsrc_t r_rsrc = row_rsrc(static_cast<const uint8_t*>(a.dres) + at, a.dres ? bytes : 0u);
#pragma unroll
    for (int j = 0; j < NV; ++j) rv[j] = row_load16(r_rsrc, off0 + j * 16 * kRowThreads);
    const float rstd = live ? a.rstd[row] : 0.0f;

    float xh[NV][E];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (CKPT) decode_vec<E>(hc[j], hs[j], xh[j]);
      else vec_widen<XT>(hv[j], xh[j]);
      float p = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xh[j][e] *= rstd;
        const float d = vec_elem<XT>(dy[j], e);
        const float tt = a.weight ? d * vec_elem<XT>(w[j], e) : d;
        p = fmaf(tt, xh[j][e], p);
        dw[j][e] = fmaf(d, xh[j][e], dw[j][e]);
      }
      dot += p;
    }
    const float c = row_sum_f32<WPR>(dot, s_sum[parity] + grp * WPR, wave) * inv_n;
    parity ^= 1;
    const __amdgpu_buffer_rsrc_t o_rsrc = row_rsrc(static_cast<uint8_t*>(a.dx) + at, bytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = vec_elem<XT>(dy[j], e);
        const float tt = a.weight ? d * vec_elem<XT>(w[j], e) : d;
        const float n = fmaf(-xh[j][e], c, tt) * rstd;
        o[e] = a.dres ? n + vec_elem<XT>(rv[j], e) : n;
      }
      row_store16<0>(o_rsrc, off0 + j * 16 * kRowThreads, vec_narrow<XT>(o));
    }
  }
  if (!a.partials) return;

  // Row groups, upper half onto lower half until one is left.
#pragma unroll
  for (int half = kGroups / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (grp >= half && grp < 2 * half) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) s_part[((grp - half) * NV * E + j * E + e) * kRowThreads + t] = dw[j][e];
    }
    __syncthreads();
    if (grp < half) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[j][e] += s_part[(grp * NV * E + j * E + e) * kRowThreads + t];
    }
  }
  if (grp != 0) return;
  const __amdgpu_buffer_rsrc_t p_rsrc = row_rsrc(a.partials + (size_t)blockIdx.x * a.cols, (uint32_t)a.cols * 4u);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; e += 4)
      row_store16<0>(p_rsrc, ((t + j * kRowThreads) * E + e) * 4, vec_narrow<kF32>(dw[j] + e));
}

// Rows longer than the register form holds: dx by one workgroup of 16
// wavefronts per row, which reads the row twice, and the rows' partial dw by
// column tiles of 1024 vectors.
template <int XT, bool CKPT>
struct LongRow {
  static constexpr int E = VecTraits<XT>::kElems;
  const NormBwdArgs& a;
  int nvec, nb;
  __device__ void load(int64_t row, int i, float rstd, float* dy, float* xh) const {
    vec_widen<XT>(static_cast<const uint4*>(a.dy)[(size_t)row * nvec + i], dy);
    if constexpr (CKPT) {
      uint32_t w[E / 4];
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.cq + (size_t)row * a.cols + (size_t)i * E);
#pragma unroll
      for (int d = 0; d < E / 4; ++d) w[d] = p[d];
      decode_vec<E>(w, a.cs[(size_t)row * nb + i / (a.cblock / E)], xh);
    } else {
      vec_widen<XT>(static_cast<const uint4*>(a.h)[(size_t)row * nvec + i], xh);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) xh[e] *= rstd;
  }
};

template <int XT, bool CKPT>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_dx_long_kernel(NormBwdArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  __shared__ float s_sum[2][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const LongRow<XT, CKPT> lr{a, a.cols / E, CKPT ? (a.cols + a.cblock - 1) / a.cblock : 0};
  const uint4* wv = static_cast<const uint4*>(a.weight);
  const float inv_n = 1.0f / (float)a.cols;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int i = threadIdx.x; i < lr.nvec; i += 1024) {
      float dy[E], xh[E], p = 0.0f;
      lr.load(row, i, rstd, dy, xh);
      const uint4 w = wv ? wv[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < E; ++e) p = fmaf(wv ? dy[e] * vec_elem<XT>(w, e) : dy[e], xh[e], p);
      dot += p;
    }
    const float c = row_sum_f32<16>(dot, s_sum[parity], wave) * inv_n;
    parity ^= 1;
    for (int i = threadIdx.x; i < lr.nvec; i += 1024) {
      float dy[E], xh[E], o[E];
      lr.load(row, i, rstd, dy, xh);
      const uint4 w = wv ? wv[i] : make_uint4(0u, 0u, 0u, 0u);
      const uint4 rv = a.dres ? static_cast<const uint4*>(a.dres)[(size_t)row * lr.nvec + i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float n = fmaf(-xh[e], c, wv ? dy[e] * vec_elem<XT>(w, e) : dy[e]) * rstd;
        o[e] = a.dres ? n + vec_elem<XT>(rv, e) : n;
      }
      static_cast<uint4*>(a.dx)[(size_t)row * lr.nvec + i] = vec_narrow<XT>(o);
    }
  }
}

template <int XT, bool CKPT>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_dw_long_kernel(NormBwdArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  const LongRow<XT, CKPT> lr{a, a.cols / E, CKPT ? (a.cols + a.cblock - 1) / a.cblock : 0};
  const int i = blockIdx.x * 1024 + threadIdx.x;
  if (i >= lr.nvec) return;
  float dw[E];
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float dy[E], xh[E];
    lr.load(row, i, a.rstd[row], dy, xh);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = fmaf(dy[e], xh[e], dw[e]);
  }
  float* p = a.partials + (size_t)blockIdx.y * a.cols + (size_t)i * E;
#pragma unroll
  for (int e = 0; e < E; ++e) p[e] = dw[e];
}

// ---------------------------------------------------------------------------
// sums of partial rows
// ---------------------------------------------------------------------------
// out[c] = sum_p partials[p][c]: 64 columns per workgroup, wavefront w takes
// the partial rows w, w + 16, ..., and the 16 sums are added in order. With no
// partial rows the sums are zero. 2.4 us for 256 x 4096 (the partials come from the
// caches they were just written to).
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* __restrict__ partials, int parts, int cols,
                                                           float* __restrict__ out) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < cols; c0 += (int64_t)gridDim.x * 64) {
    const int64_t c = c0 + lane;
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 8
      for (int p = wave; p < parts; p += 16) v += partials[(size_t)p * cols + c];
    }
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < cols) {
      float t = s[0][lane];
#pragma unroll
      for (int i = 1; i < 16; ++i) t += s[i][lane];
      out[c] = t;
    }
    __syncthreads();
  }
}

hipError_t launch_column_sums(const float* partials, int parts, int cols, float* out, hipStream_t st) {
  const int64_t want = ((int64_t)cols + 63) / 64;
  hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)(want < (1 << 20) ? want : 1 << 20)), dim3(1024), 0, st, partials,
                     parts, cols, out);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// Workgroups beyond this many walk over several rows (a launch holds fewer than
// 2^32 threads).
constexpr int64_t kMaxRowBlocks = 1 << 20;

template <int XT, int WPR, int NV>
static hipError_t launch_norm_t(const NormArgs& a, hipStream_t st) {
  using C = NormFwd<XT, WPR, NV>;
  const int64_t want = ((int64_t)a.rows + C::kRows - 1) / C::kRows;
  hipLaunchKernelGGL((rmsnorm_quant_kernel<XT, WPR, NV>), dim3((unsigned)(want < kMaxRowBlocks ? want : kMaxRowBlocks)),
                     dim3(C::kThreads), 0, st, a);
  return hipGetLastError();
}

// Wavefronts per row and vectors per thread. A workgroup per row (or four) leaves
// the overlap of one row's latency with another's traffic to the scheduler:
// 16384 x 4096 bf16 with residual and checkpoint takes 93.6 us (5.8 TB/s) with
// 4 x 2 that way, 106 us with a grid of 4 workgroups per CU that walk over the
// rows, and 113 us with one wavefront per row and 8 vectors, whose registers hold
// two wavefronts per SIMD. Where two forms serve one width the first is for few
// rows, whose latency counts (us, 7168 columns: one row 3.9 with 8 x 2 and 4.7
// with 4 x 4, 4681 rows 53.2 and 51.1; 2048 columns: 1000 rows 4.8 with 4 x 1 and
// 5.4 with 1 x 4, 16384 rows 53.0 and 49.3).
template <int XT>
static hipError_t launch_norm_x(const NormArgs& a, hipStream_t st) {
  const int nvec = a.cols / VecTraits<XT>::kElems;
  if (nvec <= 64 * 1) return launch_norm_t<XT, 1, 1>(a, st);
  if (nvec <= 64 * 2) return launch_norm_t<XT, 1, 2>(a, st);
  if (nvec <= 64 * 4) return a.rows < 4096 ? launch_norm_t<XT, 4, 1>(a, st) : launch_norm_t<XT, 1, 4>(a, st);
  if (nvec <= 256 * 2) return launch_norm_t<XT, 4, 2>(a, st);
  if (nvec <= 256 * 4) return a.rows < 1024 ? launch_norm_t<XT, 8, 2>(a, st) : launch_norm_t<XT, 4, 4>(a, st);
  if (nvec <= 512 * 4) return launch_norm_t<XT, 8, 4>(a, st);
  if (nvec <= 1024 * 4) return launch_norm_t<XT, 16, 4>(a, st);
  hipLaunchKernelGGL((rmsnorm_quant_long_kernel<XT>), dim3((unsigned)(a.rows < kMaxRowBlocks ? a.rows : kMaxRowBlocks)),
                     dim3(1024), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_quant(const NormArgs& a, int xt, hipStream_t st) {
  return xt == kBF16 ? launch_norm_x<kBF16>(a, st) : launch_norm_x<kF32>(a, st);
}

// dw without partial sums: few rows per slot, and tensors that the caches hold.
// Measured (us, direct / partial sums; bf16, checkpoint): 130 x 4096 4.0 / 7.5,
// 512 x 4096 7.0 / 8.7, 1000 x 1024 9.7 / 8.5.
constexpr int kDirectRows = 512;
constexpr int64_t kDirectBytes = 4 << 20;

// Rows a workgroup of the backward pass takes at once, and whether the row fits
// its registers: the workspace query and the launch agree through this.
struct BwdPlan {
  int wpr, nv, parts;
  bool direct;  // dw by workgroups of the same launch
};
static BwdPlan bwd_plan(int rows, int cols, int xt) {
  const int nvec = cols / (xt == kBF16 ? 8 : 4);
  BwdPlan p{};
  if (nvec <= 64) p.wpr = 1, p.nv = 1;
  else if (nvec <= 256) p.wpr = 4, p.nv = 1;
  else if (nvec <= 512) p.wpr = 4, p.nv = 2;
  else if (nvec <= 1024) p.wpr = 16, p.nv = 1;
  else if (nvec <= 2048) p.wpr = 16, p.nv = 2;
  else p.wpr = 0;
  const int groups = p.wpr ? 16 / p.wpr : 1;
  const int64_t want = ((int64_t)rows + groups - 1) / groups;
  p.parts = (int)(want < kNumCUs ? want : kNumCUs);
  p.direct = p.wpr && rows <= kDirectRows && (int64_t)rows * cols * (xt == kBF16 ? 2 : 4) <= kDirectBytes;
  return p;
}

size_t rmsnorm_bwd_workspace_bytes(int rows, int cols, int xt) {
  return (size_t)bwd_plan(rows, cols, xt).parts * (size_t)cols * 4;
}

template <int XT, bool CKPT>
static hipError_t launch_norm_bwd_t(NormBwdArgs a, hipStream_t st) {
  const BwdPlan p = bwd_plan(a.rows, a.cols, XT);
  const int nvec = a.cols / VecTraits<XT>::kElems;
  const dim3 block(1024);
  const int dw_blocks = a.dw && p.direct ? (nvec + kColVecs - 1) / kColVecs : 0;
  if (dw_blocks) a.partials = nullptr;
  const bool dw_first = dw_blocks && a.dx == a.dy;
#define HQ_LAUNCH(WPR, NV)                                                                                               \
  do {                                                                                                                   \
    if (dw_first)                                                                                                        \
      hipLaunchKernelGGL((rmsnorm_bwd_kernel<XT, WPR, NV, CKPT>), dim3(dw_blocks), block, 0, st, a, 0);                  \
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<XT, WPR, NV, CKPT>), dim3(p.parts + (dw_first ? 0 : dw_blocks)), block, 0, st, \
                       a, p.parts);                                                                                      \
  } while (0)
  if (p.wpr == 1) HQ_LAUNCH(1, 1);
  else if (p.wpr == 4 && p.nv == 1) HQ_LAUNCH(4, 1);
  else if (p.wpr == 4) HQ_LAUNCH(4, 2);
  else if (p.wpr == 16 && p.nv == 1) HQ_LAUNCH(16, 1);
  else if (p.wpr == 16) HQ_LAUNCH(16, 2);
  else {
    // dw first: dx may be dy's own buffer
    if (a.partials) {
      hipLaunchKernelGGL((rmsnorm_bwd_dw_long_kernel<XT, CKPT>), dim3((nvec + 1023) / 1024, p.parts), block, 0, st, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((rmsnorm_bwd_dx_long_kernel<XT, CKPT>), dim3(a.rows < kNumCUs * 2 ? a.rows : kNumCUs * 2), block, 0,
                       st, a);
  }
#undef HQ_LAUNCH
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.partials) return e;
  return launch_column_sums(a.partials, p.parts, a.cols, a.dw, st);
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int xt, hipStream_t st) {
  if (a.rows == 0) return a.dw ? launch_column_sums(nullptr, 0, a.cols, a.dw, st) : hipSuccess;
  if (xt == kBF16) return a.cq ? launch_norm_bwd_t<kBF16, true>(a, st) : launch_norm_bwd_t<kBF16, false>(a, st);
  return a.cq ? launch_norm_bwd_t<kF32, true>(a, st) : launch_norm_bwd_t<kF32, false>(a, st);
}

}  // namespace hq
