// RMS norm and layer norm with the residual's addition and FP8 output, and their
// backward passes, gfx950.
//
//   forward   h = x + residual            rstd = 1 / sqrt(mean_c h^2 + eps)
//             y = (h * rstd) * w          s = max(amax_row(y) / fmax, 2^-126)
//             q = cast(y * (1 / s))       optionally h itself and an 8-bit block-wise checkpoint of it
//   backward  xh = h * rstd, t = dy * w   dx = dres + rstd * (t - xh * mean_c(t * xh))
//             dw = sum_rows dy * xh
//
// Layer norm (LN) has d = h - mean_c h in h's place, and a bias:
//   forward   rstd = 1 / sqrt(mean_c d^2 + eps), y = (d * rstd) * w + b
//   backward  xh = d * rstd, dx = dres + rstd * (t - mean_c t - xh * mean_c(t * xh)), db = sum_rows dy
// Its sum of squares is taken of the differences, which the registers hold by then
// (one more exchange across a row's wavefronts): sums of h and h^2 in one go cancel
// where a row's mean is large beside its deviation. For the same reason the mean is
// corrected by the mean of these differences, summed in the same exchange: the sum of
// h is off by roundings of the mean's size, which may pass the deviation's (of constant
// float32 rows of 1040, 12345.678 came out as -0.3 and -7.7e7 as -1). Without / with the
// correction, bf16 with residual, h and copy, us in graphs: 1 x 7168 4.9 / 5.0, 1000 x 7168
// 11.2 / 11.9, 16384 x 4096 84.2 / 85.2, 4096 x 16384 105.8 / 109.5, 2048 x 32768 136 / 118.
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

// A layer norm's differences d = h - mean from their sum and that of their squares: the
// mean's correction c = mean_c d, 0 where it is no number (rows whose codes are NaN
// anyway), and sum (d - c)^2 = sum d^2 - c sum d. c is some units in the mean's last place,
// so that this cancels in rows alone that are constant but for as much, and gives 0 exactly
// in a constant one.
__device__ __forceinline__ float mean_correction(float sum_d, int cols, float& sum_dd) {
  float c = sum_d / (float)cols;
  c = fabsf(c) < __builtin_inff() ? c : 0.0f;
  if (sum_dd < __builtin_inff()) sum_dd = fmaxf(fmaf(-sum_d, c, sum_dd), 0.0f);
  return c;
}

template <bool LN, int XT, int WPR, int NV>
__global__ __launch_bounds__((NormFwd<XT, WPR, NV>::kThreads)) void norm_quant_kernel(NormArgs a) {
  using C = NormFwd<XT, WPR, NV>;
  constexpr int E = C::E;
  static_assert(WPR == 1 || C::kRows == 1, "one row per workgroup where a row needs its barrier");
  __shared__ float s_sum[WPR], s_mean[LN ? WPR : 1], s_diff[LN ? WPR : 1];
  __shared__ uint32_t s_max[WPR], s_fin[WPR];
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % WPR);
  const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x / C::kRowThreads);
  const int t = threadIdx.x % C::kRowThreads;
  const uint32_t row_bytes = (uint32_t)a.cols * (16 / E);
  const int off0 = t * 16;             // byte offset of vector 0 in a row; a step adds 16 kRowThreads
  const int nb = a.cblock ? (a.cols + a.cblock - 1) / a.cblock : 0;
  const int g = a.cblock / E;
  const float inv_n = 1.0f / (float)a.cols;

  uint4 w[NV], b[LN ? NV : 1];
  const __amdgpu_buffer_rsrc_t w_rsrc = row_rsrc(a.weight, a.weight ? row_bytes : 0u);
  const __amdgpu_buffer_rsrc_t b_rsrc = row_rsrc(a.bias, LN && a.bias ? row_bytes : 0u);
  auto load_affine = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j) w[j] = row_load16(w_rsrc, off0 + j * 16 * C::kRowThreads);
    if constexpr (LN) {
#pragma unroll
      for (int j = 0; j < NV; ++j) b[j] = row_load16(b_rsrc, off0 + j * 16 * C::kRowThreads);
    }
  };
  // A layer norm of 16-bit rows with several vectors per thread fetches weight and bias
  // with each row, after its sum: held over the row's loads they cost a wavefront per SIMD or
  // two, or spills. With residual, h and copy, us in graphs over one set of tensors (whose part
  // in the Infinity Cache makes the large ones faster than HBM alone), held / fetched: 16384 x 4096
  // 88.3 / 85.8, 8192 x 7168 86.1 / 76.0, 16384 x 2048 47.5 / 44.4, 2048 x 32768 292 / 118;
  // 16384 x 1024 23.1 / 23.8 and float32 8192 x 4096 71.3 / 73.9, which hold them.
  constexpr bool kLate = LN && XT == kBF16 && NV >= 2 && WPR * NV > 2;
  if constexpr (!kLate) load_affine();

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
      for (int e = 0; e < E; ++e) ss[j] = LN ? ss[j] + v[j][e] : fmaf(v[j][e], v[j][e], ss[j]);
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
    float mean = 0.0f, total;
    if constexpr (LN) {
      if constexpr (kLate) {
        __builtin_amdgcn_sched_barrier(0);
        load_affine();
        __builtin_amdgcn_sched_barrier(0);
      }
      mean = row_sum_f32<WPR>(ss[0], s_mean, wave) / (float)a.cols;
      // past the row's end v is 0 and stays 0
      auto inside = [&](int j) { return (t + j * C::kRowThreads) * E < a.cols; };
      float sd[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        ss[j] = sd[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[j][e] -= inside(j) ? mean : 0.0f;
          sd[j] += v[j][e];
          ss[j] = fmaf(v[j][e], v[j][e], ss[j]);
        }
      }
#pragma unroll
      for (int j = 1; j < NV; ++j) {
        ss[0] += ss[j];
        sd[0] += sd[j];
      }
      float sum_d;
      row_sum2_f32<WPR>(ss[0], sd[0], s_sum, s_diff, wave, &total, &sum_d);
      const float c = mean_correction(sum_d, a.cols, total);
      mean += c;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] -= inside(j) ? c : 0.0f;
    } else {
      total = row_sum_f32<WPR>(ss[0], s_sum, wave);
    }
    const float rstd = 1.0f / sqrtf(fmaf(total, inv_n, a.eps));
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[j][e] = a.weight ? v[j][e] * rstd * vec_elem<XT>(w[j], e) : v[j][e] * rstd;
        if constexpr (LN) v[j][e] += vec_elem<XT>(b[j], e);
      }
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
      if (LN && a.mean) a.mean[row] = mean;
    }
  }
}

// Rows longer than the register form holds: one workgroup of 16 wavefronts per
// row reads the row three times (sum of squares and checkpoint, maximum, cast
// and h), for a layer norm four times (sum and checkpoint, sums of the differences
// and of their squares, ...). h is written in the last pass only, each vector after its own reads,
// so h may be the residual's or x's own buffer here too.
template <bool LN, int XT>
__global__ __launch_bounds__(1024) void norm_quant_long_kernel(NormArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  __shared__ float s_sum[16], s_mean[16], s_diff[16];
  __shared__ uint32_t s_max[16], s_fin[16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = threadIdx.x;
  const int nvec = a.cols / E;
  const int nb = a.cblock ? (a.cols + a.cblock - 1) / a.cblock : 0;
  const int g = a.cblock / E;
  const float inv_n = 1.0f / (float)a.cols;
  const uint4* wv = static_cast<const uint4*>(a.weight);
  const uint4* bv = LN ? static_cast<const uint4*>(a.bias) : nullptr;
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
      for (int e = 0; e < E; ++e) p = LN ? p + v[e] : fmaf(v[e], v[e], p);
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
    float mean = 0.0f, c = 0.0f, total;  // a layer norm's first mean and its correction
    if constexpr (LN) {
      mean = row_sum_f32<16>(ss, s_mean, wave) / (float)a.cols;
      float sd = 0.0f, sum_d;
      ss = 0.0f;
      for (int i = t; i < nvec; i += 1024) {
        float v[E], p = 0.0f, q = 0.0f;
        load_h(i, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          p = fmaf(v[e] - mean, v[e] - mean, p);
          q += v[e] - mean;
        }
        ss += p;
        sd += q;
      }
      row_sum2_f32<16>(ss, sd, s_sum, s_diff, wave, &total, &sum_d);
      c = mean_correction(sum_d, a.cols, total);
    } else {
      total = row_sum_f32<16>(ss, s_sum, wave);
    }
    const float rstd = 1.0f / sqrtf(fmaf(total, inv_n, a.eps));
    auto load_y = [&](int i, float* h, float* y) {
      load_h(i, h);
      const uint4 w = wv ? wv[i] : make_uint4(0u, 0u, 0u, 0u);
      const uint4 b = LN && bv ? bv[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = LN ? h[e] - mean - c : h[e];
        y[e] = wv ? d * rstd * vec_elem<XT>(w, e) : d * rstd;
        if constexpr (LN) y[e] += vec_elem<XT>(b, e);
      }
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
      if (LN && a.mean) a.mean[row] = mean + c;
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
template <bool LN, int XT, bool CKPT>
__device__ __forceinline__ void norm_dw_columns(const NormBwdArgs& a, int tile, float* s) {
  constexpr int E = VecTraits<XT>::kElems;
  const int i = tile * kColVecs + (threadIdx.x & 7);  // vector column
  const int nvec = a.cols / E;
  const int nb = CKPT ? (a.cols + a.cblock - 1) / a.cblock : 0;
  const int gsh = CKPT ? __builtin_ctz(a.cblock / E) : 0;
  constexpr int N = LN ? 2 * E : E;  // dw's sums, then db's
  float dw[N];
#pragma unroll
  for (int e = 0; e < N; ++e) dw[e] = 0.0f;
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
      const float mean = LN ? a.mean[row] : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dw[e] = fmaf(vec_elem<XT>(dy, e), (LN ? xh[e] - mean : xh[e]) * rstd, dw[e]);
        if constexpr (LN) dw[E + e] += vec_elem<XT>(dy, e);
      }
    }
  }
  if (!slots_sum<N>(dw, s) || i >= nvec) return;
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    float* out = e < E ? a.dw : a.db;
    if (out) *reinterpret_cast<float4*>(out + (size_t)i * E + e % E) = make_float4(dw[e], dw[e + 1], dw[e + 2], dw[e + 3]);
  }
}

template <bool LN, int XT, int WPR, int NV, bool CKPT>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdArgs a, int row_blocks) {
  constexpr int E = VecTraits<XT>::kElems;
  constexpr int kRowThreads = 64 * WPR;
  constexpr int kGroups = 16 / WPR;
  constexpr int kCols = kRowThreads * NV * E;
  static_assert(kGroups == 1 || kCols * (kGroups / 2) <= kBwdLdsFloats, "row groups meet in LDS");
  constexpr int kPart = kGroups > 1 ? kCols * (kGroups / 2) : 1;
  constexpr int kSlots = 16 * 8 * (LN ? 2 * E : E);  // of norm_dw_columns
  __shared__ float s_part[kPart < kSlots ? kSlots : kPart];
  __shared__ float s_sum[2][16], s_mean[2][LN ? 16 : 1];
  if ((int)blockIdx.x >= row_blocks) return norm_dw_columns<LN, XT, CKPT>(a, blockIdx.x - row_blocks, s_part);
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
  float dw[NV][E], db[LN ? NV : 1][E];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      dw[j][e] = 0.0f;
      if constexpr (LN) db[j][e] = 0.0f;
    }

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
    const float mean = LN && live ? a.mean[row] : 0.0f;

    float xh[NV][E];
    float dot = 0.0f, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (CKPT) decode_vec<E>(hc[j], hs[j], xh[j]);
      else vec_widen<XT>(hv[j], xh[j]);
      float p = 0.0f, q = 0.0f;
      // past the row's end, where h reads 0, nothing may pass float32's range: dy's 0 times it
      const float m = (t + j * kRowThreads) * E < a.cols ? mean : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xh[j][e] = LN ? (xh[j][e] - m) * rstd : xh[j][e] * rstd;
        const float d = vec_elem<XT>(dy[j], e);
        const float tt = a.weight ? d * vec_elem<XT>(w[j], e) : d;
        p = fmaf(tt, xh[j][e], p);
        dw[j][e] = fmaf(d, xh[j][e], dw[j][e]);
        if constexpr (LN) {
          q += tt;
          db[j][e] += d;
        }
      }
      dot += p;
      if constexpr (LN) sum += q;
    }
    float c, c0 = 0.0f;
    if constexpr (LN) {
      row_sum2_f32<WPR>(dot, sum, s_sum[parity] + grp * WPR, s_mean[parity] + grp * WPR, wave, &c, &c0);
      c *= inv_n;
      c0 *= inv_n;
    } else {
      c = row_sum_f32<WPR>(dot, s_sum[parity] + grp * WPR, wave) * inv_n;
    }
    parity ^= 1;
    const __amdgpu_buffer_rsrc_t o_rsrc = row_rsrc(static_cast<uint8_t*>(a.dx) + at, bytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = vec_elem<XT>(dy[j], e);
        const float tt = a.weight ? d * vec_elem<XT>(w[j], e) : d;
        const float n = fmaf(-xh[j][e], c, LN ? tt - c0 : tt) * rstd;
        o[e] = a.dres ? n + vec_elem<XT>(rv[j], e) : n;
      }
      row_store16<0>(o_rsrc, off0 + j * 16 * kRowThreads, vec_narrow<XT>(o));
    }
  }
  if (!a.partials) return;

  // Row groups, upper half onto lower half until one is left; `part` is the
  // workgroup's partial row of these sums.
  auto write_sums = [&](float (&sums)[NV][E], float* part) {
#pragma unroll
    for (int half = kGroups / 2; half >= 1; half /= 2) {
      __syncthreads();
      if (grp >= half && grp < 2 * half) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < E; ++e) s_part[((grp - half) * NV * E + j * E + e) * kRowThreads + t] = sums[j][e];
      }
      __syncthreads();
      if (grp < half) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < E; ++e) sums[j][e] += s_part[(grp * NV * E + j * E + e) * kRowThreads + t];
      }
    }
    if (grp != 0) return;
    const __amdgpu_buffer_rsrc_t p_rsrc = row_rsrc(part, (uint32_t)a.cols * 4u);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < E; e += 4)
        row_store16<0>(p_rsrc, ((t + j * kRowThreads) * E + e) * 4, vec_narrow<kF32>(sums[j] + e));
  };
  float* part = a.partials + (size_t)blockIdx.x * a.cols * (LN ? 2 : 1);
  write_sums(dw, part);
  if constexpr (LN) write_sums(db, part + a.cols);
}

// Rows longer than the register form holds: dx by one workgroup of 16
// wavefronts per row, which reads the row twice, and the rows' partial dw by
// column tiles of 1024 vectors.
template <bool LN, int XT, bool CKPT>
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
    const float mean = LN ? a.mean[row] : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) xh[e] = LN ? (xh[e] - mean) * rstd : xh[e] * rstd;
  }
};

template <bool LN, int XT, bool CKPT>
__global__ __launch_bounds__(1024) void norm_bwd_dx_long_kernel(NormBwdArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  __shared__ float s_sum[2][16], s_mean[2][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const LongRow<LN, XT, CKPT> lr{a, a.cols / E, CKPT ? (a.cols + a.cblock - 1) / a.cblock : 0};
  const uint4* wv = static_cast<const uint4*>(a.weight);
  const float inv_n = 1.0f / (float)a.cols;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float dot = 0.0f, sum = 0.0f;
    for (int i = threadIdx.x; i < lr.nvec; i += 1024) {
      float dy[E], xh[E], p = 0.0f, q = 0.0f;
      lr.load(row, i, rstd, dy, xh);
      const uint4 w = wv ? wv[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float tt = wv ? dy[e] * vec_elem<XT>(w, e) : dy[e];
        p = fmaf(tt, xh[e], p);
        if constexpr (LN) q += tt;
      }
      dot += p;
      if constexpr (LN) sum += q;
    }
    float c, c0 = 0.0f;
    if constexpr (LN) {
      row_sum2_f32<16>(dot, sum, s_sum[parity], s_mean[parity], wave, &c, &c0);
      c *= inv_n;
      c0 *= inv_n;
    } else {
      c = row_sum_f32<16>(dot, s_sum[parity], wave) * inv_n;
    }
    parity ^= 1;
    for (int i = threadIdx.x; i < lr.nvec; i += 1024) {
      float dy[E], xh[E], o[E];
      lr.load(row, i, rstd, dy, xh);
      const uint4 w = wv ? wv[i] : make_uint4(0u, 0u, 0u, 0u);
      const uint4 rv = a.dres ? static_cast<const uint4*>(a.dres)[(size_t)row * lr.nvec + i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float tt = wv ? dy[e] * vec_elem<XT>(w, e) : dy[e];
        const float n = fmaf(-xh[e], c, LN ? tt - c0 : tt) * rstd;
        o[e] = a.dres ? n + vec_elem<XT>(rv, e) : n;
      }
      static_cast<uint4*>(a.dx)[(size_t)row * lr.nvec + i] = vec_narrow<XT>(o);
    }
  }
}

template <bool LN, int XT, bool CKPT>
__global__ __launch_bounds__(1024) void norm_bwd_dw_long_kernel(NormBwdArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  const LongRow<LN, XT, CKPT> lr{a, a.cols / E, CKPT ? (a.cols + a.cblock - 1) / a.cblock : 0};
  const int i = blockIdx.x * 1024 + threadIdx.x;
  if (i >= lr.nvec) return;
  float dw[E], db[E];
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = db[e] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float dy[E], xh[E];
    lr.load(row, i, a.rstd[row], dy, xh);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      dw[e] = fmaf(dy[e], xh[e], dw[e]);
      if constexpr (LN) db[e] += dy[e];
    }
  }
  float* p = a.partials + (size_t)blockIdx.y * a.cols * (LN ? 2 : 1) + (size_t)i * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    p[e] = dw[e];
    if constexpr (LN) p[(size_t)a.cols + e] = db[e];
  }
}

// ---------------------------------------------------------------------------
// sums of partial rows
// ---------------------------------------------------------------------------
// out[c] = sum_p partials[p][c]: 64 columns per workgroup, wavefront w takes
// the partial rows w, w + 16, ..., and the 16 sums are added in order. With no
// partial rows the sums are zero. 2.4 us for 256 x 4096 (the partials come from the
// caches they were just written to). The columns from `split` on go to `out2`; an
// output that is null is left out.
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* __restrict__ partials, int parts, int64_t cols,
                                                           float* __restrict__ out, float* __restrict__ out2, int64_t split) {
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
      if (c < split) {
        if (out) out[c] = t;
      } else if (out2) {
        out2[c - split] = t;
      }
    }
    __syncthreads();
  }
}

static hipError_t column_sums(const float* partials, int parts, int64_t cols, float* out, float* out2, int64_t split,
                              hipStream_t st) {
  const int64_t want = (cols + 63) / 64;
  hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)(want < (1 << 20) ? want : 1 << 20)), dim3(1024), 0, st, partials,
                     parts, cols, out, out2, split);
  return hipGetLastError();
}
hipError_t launch_column_sums(const float* partials, int parts, int cols, float* out, hipStream_t st) {
  return column_sums(partials, parts, cols, out, nullptr, cols, st);
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// Workgroups beyond this many walk over several rows (a launch holds fewer than
// 2^32 threads).
constexpr int64_t kMaxRowBlocks = 1 << 20;

template <bool LN, int XT, int WPR, int NV>
static hipError_t launch_norm_t(const NormArgs& a, hipStream_t st) {
  using C = NormFwd<XT, WPR, NV>;
  const int64_t want = ((int64_t)a.rows + C::kRows - 1) / C::kRows;
  hipLaunchKernelGGL((norm_quant_kernel<LN, XT, WPR, NV>), dim3((unsigned)(want < kMaxRowBlocks ? want : kMaxRowBlocks)),
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
// 5.4 with 1 x 4, 16384 rows 53.0 and 49.3). The form of 16 x 4 spills with bf16 rows,
// 100 bytes a lane for an RMS norm and 16 for a layer norm; the backward pass's of 16 x 2
// for a layer norm alone, 24 bytes and 60 from the copy.
template <bool LN, int XT>
static hipError_t launch_norm_x(const NormArgs& a, hipStream_t st) {
  const int nvec = a.cols / VecTraits<XT>::kElems;
  if (nvec <= 64 * 1) return launch_norm_t<LN, XT, 1, 1>(a, st);
  if (nvec <= 64 * 2) return launch_norm_t<LN, XT, 1, 2>(a, st);
  if (nvec <= 64 * 4) return a.rows < 4096 ? launch_norm_t<LN, XT, 4, 1>(a, st) : launch_norm_t<LN, XT, 1, 4>(a, st);
  if (nvec <= 256 * 2) return launch_norm_t<LN, XT, 4, 2>(a, st);
  if (nvec <= 256 * 4) return a.rows < 1024 ? launch_norm_t<LN, XT, 8, 2>(a, st) : launch_norm_t<LN, XT, 4, 4>(a, st);
  if (nvec <= 512 * 4) return launch_norm_t<LN, XT, 8, 4>(a, st);
  if (nvec <= 1024 * 4) return launch_norm_t<LN, XT, 16, 4>(a, st);
  hipLaunchKernelGGL((norm_quant_long_kernel<LN, XT>), dim3((unsigned)(a.rows < kMaxRowBlocks ? a.rows : kMaxRowBlocks)),
                     dim3(1024), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_quant(const NormArgs& a, int xt, hipStream_t st) {
  return xt == kBF16 ? launch_norm_x<false, kBF16>(a, st) : launch_norm_x<false, kF32>(a, st);
}

hipError_t launch_layernorm_quant(const NormArgs& a, int xt, hipStream_t st) {
  return xt == kBF16 ? launch_norm_x<true, kBF16>(a, st) : launch_norm_x<true, kF32>(a, st);
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
size_t layernorm_bwd_workspace_bytes(int rows, int cols, int xt) { return 2 * rmsnorm_bwd_workspace_bytes(rows, cols, xt); }

template <bool LN, int XT, bool CKPT>
static hipError_t launch_norm_bwd_t(NormBwdArgs a, hipStream_t st) {
  const BwdPlan p = bwd_plan(a.rows, a.cols, XT);
  const int nvec = a.cols / VecTraits<XT>::kElems;
  const dim3 block(1024);
  const int dw_blocks = (a.dw || a.db) && p.direct ? (nvec + kColVecs - 1) / kColVecs : 0;
  if (dw_blocks) a.partials = nullptr;
  const bool dw_first = dw_blocks && a.dx == a.dy;
#define HQ_LAUNCH(WPR, NV)                                                                                               \
  do {                                                                                                                   \
    if (dw_first)                                                                                                        \
      hipLaunchKernelGGL((norm_bwd_kernel<LN, XT, WPR, NV, CKPT>), dim3(dw_blocks), block, 0, st, a, 0);                  \
    hipLaunchKernelGGL((norm_bwd_kernel<LN, XT, WPR, NV, CKPT>), dim3(p.parts + (dw_first ? 0 : dw_blocks)), block, 0, st, \
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
      hipLaunchKernelGGL((norm_bwd_dw_long_kernel<LN, XT, CKPT>), dim3((nvec + 1023) / 1024, p.parts), block, 0, st, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((norm_bwd_dx_long_kernel<LN, XT, CKPT>), dim3(a.rows < kNumCUs * 2 ? a.rows : kNumCUs * 2), block, 0,
                       st, a);
  }
#undef HQ_LAUNCH
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.partials) return e;
  return column_sums(a.partials, p.parts, (LN ? 2 : 1) * (int64_t)a.cols, a.dw, a.db, a.cols, st);
}

template <bool LN>
static hipError_t launch_norm_bwd(const NormBwdArgs& a, int xt, hipStream_t st) {
  if (a.rows == 0) return a.dw || a.db ? column_sums(nullptr, 0, (LN ? 2 : 1) * (int64_t)a.cols, a.dw, a.db, a.cols, st) : hipSuccess;
  if (xt == kBF16) return a.cq ? launch_norm_bwd_t<LN, kBF16, true>(a, st) : launch_norm_bwd_t<LN, kBF16, false>(a, st);
  return a.cq ? launch_norm_bwd_t<LN, kF32, true>(a, st) : launch_norm_bwd_t<LN, kF32, false>(a, st);
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int xt, hipStream_t st) { return launch_norm_bwd<false>(a, xt, st); }
hipError_t launch_layernorm_bwd(const NormBwdArgs& a, int xt, hipStream_t st) { return launch_norm_bwd<true>(a, xt, st); }

}  // namespace hq
