// Activation into FP8 codes with an 8-bit checkpoint of its input, and the
// backward pass from that checkpoint, gfx950.
//
//   forward   a = act(z), or gated act(z1) * z2 with z = [z1 | z2]
//             s = max(amax_row(a) / fmax, 2^-126), q = cast(a * (1 / s))
//             zq, zs: block-wise E4M3 of z (the rule and layout of hq_quantize_fp8_blockwise)
//   backward  z^ = dec(zq) * zs
//             dz = da * act'(z^), or gated [da * z2^ * act'(z1^) | da * act(z1^)]
//             db = sum_rows dz
#include "hq_act.h"
#include "hq_launch.h"
#include "hq_row.h"

namespace hq {

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Thread t of a row's WPR wavefronts owns vectors t, t + 64 WPR, ... (gated: of
// both halves); the activated values stay in registers between the row's
// maximum and the cast.
template <int XT, int WPR, int ACT, bool GATED>
struct ActFwd {
  static constexpr int E = VecTraits<XT>::kElems;
  static constexpr int kRowThreads = 64 * WPR;
  static constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
  static constexpr int kThreads = kRowThreads * kRows;

  // values of one vector of z: its checkpoint, and the activated values
  static __device__ __forceinline__ void vec(const ActArgs& a, const uint4& z1, const uint4& z2, int64_t row, int i,
                                             float* out) {
    float f1[E], f2[E];
    vec_widen<XT>(z1, f1);
    if constexpr (GATED) vec_widen<XT>(z2, f2);
    if (a.cblock) {
      const int wide = GATED ? 2 * a.cols : a.cols;
      const int nb = (wide + a.cblock - 1) / a.cblock, g = a.cblock / E;
      const __amdgpu_buffer_rsrc_t c1 = row_rsrc(a.cq + (size_t)row * wide, (uint32_t)a.cols);
      const __amdgpu_buffer_rsrc_t s1 = row_rsrc(a.cs + (size_t)row * nb, (uint32_t)(GATED ? nb / 2 : nb) * 4u);
      uint32_t w[E / 4];
      float s = checkpoint_vec<E>(f1, g, w);
      row_store_codes<E, kStreamPolicy>(c1, i * E, w);
      if ((i & (g - 1)) == 0) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), s1, i / g * 4, 0, 0);
      if constexpr (GATED) {
        const __amdgpu_buffer_rsrc_t c2 = row_rsrc(a.cq + (size_t)row * wide + a.cols, (uint32_t)a.cols);
        const __amdgpu_buffer_rsrc_t s2 = row_rsrc(a.cs + (size_t)row * nb + nb / 2, (uint32_t)(nb / 2) * 4u);
        s = checkpoint_vec<E>(f2, g, w);
        row_store_codes<E, kStreamPolicy>(c2, i * E, w);
        if ((i & (g - 1)) == 0) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), s2, i / g * 4, 0, 0);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = GATED ? act_value<ACT>(f1[e]) * f2[e] : act_value<ACT>(f1[e]);
  }
};

template <int XT, int WPR, int NV, int ACT, bool GATED>
__global__ __launch_bounds__((ActFwd<XT, WPR, ACT, GATED>::kThreads)) void act_quant_kernel(ActArgs a) {
  using C = ActFwd<XT, WPR, ACT, GATED>;
  constexpr int E = C::E;
  static_assert(WPR == 1 || C::kRows == 1, "one row per workgroup where a row needs its barrier");
  __shared__ uint32_t s_max[2][WPR], s_fin[WPR];
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % WPR);
  const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x / C::kRowThreads);
  const int t = threadIdx.x % C::kRowThreads;
  const uint32_t half_bytes = (uint32_t)a.cols * (16 / E);
  const uint32_t row_bytes = GATED ? 2 * half_bytes : half_bytes;
  const int64_t step = (int64_t)gridDim.x * C::kRows;
  int parity = 0;
  for (int64_t row = (int64_t)blockIdx.x * C::kRows + grp; row < a.rows; row += step) {
    const uint8_t* zr = static_cast<const uint8_t*>(a.z) + (size_t)row * row_bytes;
    const __amdgpu_buffer_rsrc_t r1 = row_rsrc(zr, half_bytes);
    const __amdgpu_buffer_rsrc_t r2 = row_rsrc(zr + half_bytes, GATED ? half_bytes : 0u);
    uint4 z1[NV], z2[GATED ? NV : 1];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      z1[j] = row_load16(r1, (t + j * C::kRowThreads) * 16);
      if constexpr (GATED) z2[j] = row_load16(r2, (t + j * C::kRowThreads) * 16);
    }
    float v[NV][E];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      C::vec(a, z1[j], z2[GATED ? j : 0], row, t + j * C::kRowThreads, v[j]);
      m = max(m, absmax_raw<E>(v[j]));
    }
    m = row_max_u32<WPR>(m, s_max[parity], wave);
    parity ^= 1;
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
      uint32_t w[E / 4];
      if (a.fmt == kE4M3) cast_values<kE4M3, E>(v[j], r, special, w);
      else cast_values<kE5M2, E>(v[j], r, special, w);
      row_store_codes<E, kStreamPolicy>(q_rsrc, (t + j * C::kRowThreads) * E, w);
    }
    if (t == 0) a.scale[row] = s;
  }
}

// Rows longer than the register form holds: one workgroup of 16 wavefronts per
// row computes the activation twice, for the maximum and for the cast.
template <int XT, int ACT, bool GATED>
__global__ __launch_bounds__(1024) void act_quant_long_kernel(ActArgs a) {
  using C = ActFwd<XT, 16, ACT, GATED>;
  constexpr int E = C::E;
  __shared__ uint32_t s_max[16], s_fin[16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = threadIdx.x;
  const int nvec = a.cols / E;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint4* z = static_cast<const uint4*>(a.z) + (size_t)row * nvec * (GATED ? 2 : 1);
    uint32_t raw = 0, fin = 0;
    for (int i0 = 0; i0 < nvec; i0 += 1024) {  // every lane takes part in a block's maximum
      const int i = i0 + t;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      float v[E];
      C::vec(a, i < nvec ? z[i] : zero, GATED && i < nvec ? z[nvec + i] : zero, row, i, v);
      raw = max(raw, absmax_raw<E>(v));
      fin = max(fin, absmax_finite<E>(v));
    }
    const bool special = row_max_u32<16>(raw, s_max, wave) >= kInfBits;
    const float amax = __uint_as_float(row_max_u32<16>(fin, s_fin, wave));
    const float s = a.fmt == kE4M3 ? scale_from_amax<kE4M3>(amax) : scale_from_amax<kE5M2>(amax);
    const float r = 1.0f / s;
    ActArgs b = a;
    b.cblock = 0;  // the checkpoint is written
    for (int i = t; i < nvec; i += 1024) {
      float v[E];
      C::vec(b, z[i], GATED ? z[nvec + i] : z[i], row, i, v);
      uint32_t w[E / 4];
      if (a.fmt == kE4M3) cast_values<kE4M3, E>(v, r, special, w);
      else cast_values<kE5M2, E>(v, r, special, w);
      store_codes<E>(a.q + (size_t)row * a.cols + (size_t)i * E, w);
    }
    if (t == 0) a.scale[row] = s;
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// One vector: dz (gated: of both halves) from da and the codes, added to the sums.
template <int XT, int ACT, bool GATED>
__device__ __forceinline__ void act_bwd_vec(const uint4& dav, const uint32_t* w1, float s1, const uint32_t* w2, float s2,
                                            float* o1, float* o2, float* db) {
  constexpr int E = VecTraits<XT>::kElems;
  float z1[E], z2[E];
  decode_vec<E>(w1, s1, z1);
  if constexpr (GATED) decode_vec<E>(w2, s2, z2);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float d = vec_elem<XT>(dav, e);
    float v, g;
    act_value_grad<ACT>(z1[e], &v, &g);
    if constexpr (GATED) {
      o1[e] = d * z2[e] * g;
      o2[e] = d * v;
      db[E + e] += o2[e];
    } else {
      o1[e] = d * g;
    }
    db[e] += o1[e];
  }
}

// No row has to be seen whole, so a workgroup of 16 wavefronts takes a tile of
// 64 CW vectors of columns and walks down the rows, 16 / CW rows at a time; a
// thread keeps its columns' sums of dz in registers (unrounded), the row groups
// meet in LDS at the end, and one partial row per workgroup goes to the
// workspace for column_sums_kernel. dz goes through the caches: 8192 x 4096 bf16 SiLU
// gated (271 MB, 44.0 us at 6.15 TB/s, a large elementwise pass's best) takes 49.1 us
// replayed from a graph, 45.4 of it this kernel; 55.5 with dz streamed past them and
// two workgroups per CU; 52.6 with runs of neighbouring rows per workgroup.
template <int XT, int CW, int ACT, bool GATED>
__global__ __launch_bounds__(1024) void act_bwd_kernel(ActBwdArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  constexpr int kTileThreads = 64 * CW;
  constexpr int kGroups = 16 / CW;
  constexpr int S = GATED ? 2 * E : E;  // sums per thread
  __shared__ float s_part[S * 512];
  const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x / kTileThreads);
  const int t = threadIdx.x % kTileThreads;
  const int wide = GATED ? 2 * a.cols : a.cols;
  const int nb = (wide + a.cblock - 1) / a.cblock;
  const int gsh = __builtin_ctz(a.cblock / E);
  const int c0 = blockIdx.x * kTileThreads * E;  // first column of the tile
  const int b0 = c0 / a.cblock;                  // its first block (tiles are whole blocks)
  const uint32_t left = (uint32_t)min(a.cols - c0, kTileThreads * E);
  const uint32_t sleft = ((uint32_t)left + a.cblock - 1) / a.cblock * 4u;
  float db[S];
#pragma unroll
  for (int e = 0; e < S; ++e) db[e] = 0.0f;

  for (int64_t row = (int64_t)blockIdx.y * kGroups + grp; row < a.rows; row += (int64_t)gridDim.y * kGroups) {
    const __amdgpu_buffer_rsrc_t da_r =
        row_rsrc(static_cast<const uint8_t*>(a.da) + ((size_t)row * a.cols + c0) * (16 / E), left * (16 / E));
    const uint8_t* q1 = a.cq + (size_t)row * wide + c0;
    const float* sc1 = a.cs + (size_t)row * nb + b0;
    uint32_t w1[E / 4], w2[E / 4];
    const uint4 dav = row_load16(da_r, t * 16);
    row_load_codes<E>(row_rsrc(q1, left), t * E, w1);
    const float sz1 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row_rsrc(sc1, sleft), (t >> gsh) * 4, 0, 0));
    float sz2 = 0.0f;
    if constexpr (GATED) {
      row_load_codes<E>(row_rsrc(q1 + a.cols, left), t * E, w2);
      sz2 = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row_rsrc(sc1 + nb / 2, sleft), (t >> gsh) * 4, 0, 0));
    }
    float o1[E], o2[E];
    act_bwd_vec<XT, ACT, GATED>(dav, w1, sz1, w2, sz2, o1, o2, db);
    uint8_t* out = static_cast<uint8_t*>(a.dz) + ((size_t)row * wide + c0) * (16 / E);
    row_store16<0>(row_rsrc(out, left * (16 / E)), t * 16, vec_narrow<XT>(o1));
    if constexpr (GATED)
      row_store16<0>(row_rsrc(out + (size_t)a.cols * (16 / E), left * (16 / E)), t * 16, vec_narrow<XT>(o2));
  }
  if (!a.partials) return;

#pragma unroll
  for (int half = kGroups / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (grp >= half && grp < 2 * half) {
#pragma unroll
      for (int e = 0; e < S; ++e) s_part[((grp - half) * S + e) * kTileThreads + t] = db[e];
    }
    __syncthreads();
    if (grp < half) {
#pragma unroll
      for (int e = 0; e < S; ++e) db[e] += s_part[(grp * S + e) * kTileThreads + t];
    }
  }
  if (grp != 0) return;
  float* p = a.partials + (size_t)blockIdx.y * wide + c0;
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    const __amdgpu_buffer_rsrc_t p_rsrc = row_rsrc(p + (size_t)h * a.cols, left * 4u);
#pragma unroll
    for (int e = 0; e < E; e += 4) row_store16<0>(p_rsrc, (t * E + e) * 4, vec_narrow<kF32>(db + h * E + e));
  }
}

// Few rows: a workgroup takes 8 vector columns of every row and writes their sums
// itself, so no second launch adds partial rows.
template <int XT, int ACT, bool GATED>
__global__ __launch_bounds__(1024) void act_bwd_columns_kernel(ActBwdArgs a) {
  constexpr int E = VecTraits<XT>::kElems;
  constexpr int S = GATED ? 2 * E : E;
  __shared__ float s_sum[16 * 8 * S];
  const int i = blockIdx.x * kColVecs + (threadIdx.x & 7);  // vector column
  const int nvec = a.cols / E, wide = GATED ? 2 * a.cols : a.cols;
  const int nb = (wide + a.cblock - 1) / a.cblock;
  const int gsh = __builtin_ctz(a.cblock / E);
  float db[S];
#pragma unroll
  for (int e = 0; e < S; ++e) db[e] = 0.0f;
  if (i < nvec) {
#pragma unroll 2
    for (int row = threadIdx.x >> 3; row < a.rows; row += kColSlots) {
      const uint4 dav = static_cast<const uint4*>(a.da)[(size_t)row * nvec + i];
      uint32_t w[2][E / 4];
      float sc[2];
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(a.cq + (size_t)row * wide + h * a.cols + (size_t)i * E);
#pragma unroll
        for (int d = 0; d < E / 4; ++d) w[h][d] = p[d];
        sc[h] = a.cs[(size_t)row * nb + h * (nb / 2) + (i >> gsh)];
      }
      float o[2][E];
      act_bwd_vec<XT, ACT, GATED>(dav, w[0], sc[0], w[1], sc[1], o[0], o[1], db);
      uint4* out = static_cast<uint4*>(a.dz) + (size_t)row * (GATED ? 2 * nvec : nvec) + i;
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) out[h * nvec] = vec_narrow<XT>(o[h]);
    }
  }
  if (!a.db) return;
  if (slots_sum<S>(db, s_sum) && i < nvec) {
#pragma unroll
    for (int e = 0; e < S; e += 4)
      *reinterpret_cast<float4*>(a.db + (size_t)(e / E) * a.cols + (size_t)i * E + e % E) =
          make_float4(db[e], db[e + 1], db[e + 2], db[e + 3]);
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// Workgroups beyond this many walk over several rows.
constexpr int64_t kMaxRowBlocks = 1 << 20;

// Wavefronts per row and vectors per thread; a workgroup per row, or four, as in
// the norm (8192 x 4096 bf16 SiLU gated with checkpoint: 45.1 us, 5.3 TB/s, with 4 x 2,
// 49.0 with a grid of 4 workgroups per CU). Two forms serve one width where few
// rows and many differ (us, 2048 columns not gated: 1000 rows 4.2 with 4 x 1 and 4.7
// with 1 x 4, 16384 rows 32.8 and 27.6) and where the gated form's registers tell
// (16384 columns, 2048 rows: gated 50.3 with 8 x 4 and 57.9 with 16 x 2, not gated
// 30.2 and 27.2).
template <int XT, int ACT, bool GATED>
static hipError_t launch_act_a(const ActArgs& a, hipStream_t st) {
  const int nvec = a.cols / VecTraits<XT>::kElems;
#define HQ_LAUNCH(WPR, NV)                                                                                            \
  do {                                                                                                                \
    using C = ActFwd<XT, WPR, ACT, GATED>;                                                                            \
    const int64_t want = ((int64_t)a.rows + C::kRows - 1) / C::kRows;                                                 \
    hipLaunchKernelGGL((act_quant_kernel<XT, WPR, NV, ACT, GATED>),                                                   \
                       dim3((unsigned)(want < kMaxRowBlocks ? want : kMaxRowBlocks)), dim3(C::kThreads), 0, st, a);    \
  } while (0)
  if (nvec <= 64 * 1) HQ_LAUNCH(1, 1);
  else if (nvec <= 64 * 2) HQ_LAUNCH(1, 2);
  else if (nvec <= 64 * 4 && a.rows < 4096) HQ_LAUNCH(4, 1);
  else if (nvec <= 64 * 4) HQ_LAUNCH(1, 4);
  else if (nvec <= 256 * 2) HQ_LAUNCH(4, 2);
  else if (nvec <= 512 * 2) HQ_LAUNCH(8, 2);
  else if (nvec <= 512 * 4) {
    if constexpr (GATED || XT == kF32) HQ_LAUNCH(8, 4);
    else HQ_LAUNCH(16, 2);
  } else if (nvec <= 1024 * 4) HQ_LAUNCH(16, 4);
  else
    hipLaunchKernelGGL((act_quant_long_kernel<XT, ACT, GATED>),
                       dim3((unsigned)(a.rows < kMaxRowBlocks ? a.rows : kMaxRowBlocks)), dim3(1024), 0, st, a);
#undef HQ_LAUNCH
  return hipGetLastError();
}

template <int XT, int ACT>
static hipError_t launch_act_g(const ActArgs& a, bool gated, hipStream_t st) {
  return gated ? launch_act_a<XT, ACT, true>(a, st) : launch_act_a<XT, ACT, false>(a, st);
}

template <int XT>
static hipError_t launch_act_x(const ActArgs& a, int act, bool gated, hipStream_t st) {
  switch (act) {
    case kActRelu: return launch_act_g<XT, kActRelu>(a, gated, st);
    case kActGelu: return launch_act_g<XT, kActGelu>(a, gated, st);
    case kActGeluTanh: return launch_act_g<XT, kActGeluTanh>(a, gated, st);
    default: return launch_act_g<XT, kActSilu>(a, gated, st);
  }
}

hipError_t launch_act_quant(const ActArgs& a, int xt, int act, bool gated, hipStream_t st) {
  return xt == kBF16 ? launch_act_x<kBF16>(a, act, gated, st) : launch_act_x<kF32>(a, act, gated, st);
}

// Wavefronts across a tile, tiles across the row, row chunks: the workspace
// query and the launch agree through this.
struct ActBwdPlan {
  int cw, tiles, parts;
  bool direct;  // act_bwd_columns_kernel
};
// Measured (us, direct / partial sums; bf16): SiLU gated 130 x 4096 6.2 / 7.6,
// 300 x 1056 7.1 / 7.7, 512 x 4096 11.0 / 9.8; GELU 256 x 8192 6.9 / 8.1, 512 x 4096
// 10.0 / 7.6. The second launch costs the host another 3 us.
constexpr int kDirectRows = 384;
constexpr int64_t kDirectBytes = 4 << 20;

static ActBwdPlan act_bwd_plan(int rows, int cols, int xt) {
  const int nvec = cols / (xt == kBF16 ? 8 : 4);
  ActBwdPlan p;
  p.cw = nvec <= 64 ? 1 : 4;
  p.tiles = (nvec + 64 * p.cw - 1) / (64 * p.cw);
  const int groups = 16 / p.cw;
  const int64_t want = ((int64_t)rows + groups - 1) / groups;
  const int64_t fill = (kNumCUs + p.tiles - 1) / p.tiles;  // one workgroup per CU
  p.parts = (int)(want < fill ? want : fill);
  p.direct = rows <= kDirectRows && (int64_t)rows * cols * (xt == kBF16 ? 2 : 4) <= kDirectBytes;
  return p;
}

size_t act_bwd_workspace_bytes(int rows, int cols, int xt, bool gated) {
  return (size_t)act_bwd_plan(rows, cols, xt).parts * (size_t)cols * (gated ? 8 : 4);
}

template <int XT, int ACT, bool GATED>
static hipError_t launch_act_bwd_a(const ActBwdArgs& a, hipStream_t st) {
  const ActBwdPlan p = act_bwd_plan(a.rows, a.cols, XT);
  const dim3 grid(p.tiles, p.parts), block(1024);
  if (p.direct) {
    const int nvec = a.cols / VecTraits<XT>::kElems;
    hipLaunchKernelGGL((act_bwd_columns_kernel<XT, ACT, GATED>), dim3((nvec + kColVecs - 1) / kColVecs), block, 0, st, a);
    return hipGetLastError();
  }
  if (p.cw == 1) hipLaunchKernelGGL((act_bwd_kernel<XT, 1, ACT, GATED>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((act_bwd_kernel<XT, 4, ACT, GATED>), grid, block, 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.partials) return e;
  return launch_column_sums(a.partials, p.parts, GATED ? 2 * a.cols : a.cols, a.db, st);
}

template <int XT, int ACT>
static hipError_t launch_act_bwd_g(const ActBwdArgs& a, bool gated, hipStream_t st) {
  return gated ? launch_act_bwd_a<XT, ACT, true>(a, st) : launch_act_bwd_a<XT, ACT, false>(a, st);
}

template <int XT>
static hipError_t launch_act_bwd_x(const ActBwdArgs& a, int act, bool gated, hipStream_t st) {
  switch (act) {
    case kActRelu: return launch_act_bwd_g<XT, kActRelu>(a, gated, st);
    case kActGelu: return launch_act_bwd_g<XT, kActGelu>(a, gated, st);
    case kActGeluTanh: return launch_act_bwd_g<XT, kActGeluTanh>(a, gated, st);
    default: return launch_act_bwd_g<XT, kActSilu>(a, gated, st);
  }
}

hipError_t launch_act_bwd(const ActBwdArgs& a, int xt, int act, bool gated, hipStream_t st) {
  if (a.rows == 0) return a.db ? launch_column_sums(nullptr, 0, gated ? 2 * a.cols : a.cols, a.db, st) : hipSuccess;
  return xt == kBF16 ? launch_act_bwd_x<kBF16>(a, act, gated, st) : launch_act_bwd_x<kF32>(a, act, gated, st);
}

}  // namespace hq
