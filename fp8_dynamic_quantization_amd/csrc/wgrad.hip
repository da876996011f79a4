// Weight gradient from the FP8 codes that the forward GEMM read, gfx950:
//
//   dW[n, k] = base[n, k] + sum_m G[m, n] * x_scale[m] * dec(XQ[m, k])
//
// G bf16 [m, n], XQ uint8 [m, k], both row-major, so the contraction runs over
// the slow axis of both operands while the matrix cores want 8 consecutive
// contraction values per lane. Tiles are staged in LDS as they lie in memory
// (rows of tokens) and transposed on the way out by the LDS transpose reads:
//   ds_read_tr16_b64  16 lanes read 4 rows x 16 bf16 (lane 4r + c supplies columns
//                     4c..4c+3 of row r); lane i receives column i of the 4 rows
//   ds_read_tr8_b64   16 lanes read 8 rows x 16 bytes (lane 2r + c supplies bytes
//                     8c..8c+7 of row r); lane i receives column i of the 8 rows
// so one 8-bit and two 16-bit reads give the operands of V_MFMA_F32_16X16X32_BF16,
// whose lane l holds contraction values 8 (l / 16) .. +7 of row or column l % 16.
//
// The FP8 codes are exact in bf16 and in f16 and are converted after the read. The
// token's scale is folded into G on its way to LDS, once per workgroup. Two forms:
//   one number   v = g * scale[m] rounded to bf16, at most 2^-8 of a term: for a bf16
//                result of many tokens, over which the roundings average (2048 normal
//                tokens: 0.0016 of the result's norm beside 0.0017 from its own
//                rounding; where a column's terms cancel, more of what is left). One
//                scale for all tokens is applied to the sums instead: g and the codes
//                are exact in bf16, and no term is rounded
//   two numbers  v = hi + lo in f16, both multiplied (V_MFMA_F32_16X16X32_F16, the
//                same rate): 2^-23 of a term. f16's range is covered by scaling each
//                column of G by the power of two that takes the largest |g * scale|
//                of the column below 2^15, undone on the sums (both exact); a term
//                2^29 below its column's largest starts to lose bits, by 2^-39 of
//                that largest (half of f16's smallest step, against 2^14 or more). (Two bf16 numbers need no scaling but leave 2^-17 of a
//                term: 1.1e-6 of a result, against 6e-8 for float32 arithmetic.)
//                For a float32 result, for few tokens, which leave little to average
//                the terms' roundings over, and where the caller asks for it
//                (2048 x 4096 x 1024 bf16 50 us against 25).
#include "gemm_kernels.h"
#include "hq_row.h"

namespace hq {

typedef short wg_s4 __attribute__((ext_vector_type(4)));
typedef int wg_i2 __attribute__((ext_vector_type(2)));
typedef __bf16 wg_b8 __attribute__((ext_vector_type(8)));
typedef int wg_i4 __attribute__((ext_vector_type(4)));
#define HQ_LDS __attribute__((address_space(3)))

// BN x BK outputs per workgroup of 8 wavefronts. KS = 1: 4 wavefronts along n, 2
// along k. KS = 2: two groups of 2 x 2 wavefronts, each with its own stages, take
// the even and the odd steps of MS tokens and meet at the end.
template <int BN, int BK, int KS, int MS, bool HILO>
struct WgCfg {
  static constexpr int kThreads = 512;
  static constexpr int T = kThreads / KS;           // threads of a group
  static constexpr int kNW = KS == 1 ? 4 : 2;       // wavefronts along n
  static constexpr int kKW = 2;                     // along k
  static constexpr int WN = BN / kNW, WK = BK / kKW;
  static constexpr int FN = WN / 16, FK = WK / 16;  // fragments per wavefront
  static constexpr int kGRow = BN * 2, kXRow = BK;  // LDS row bytes
  static constexpr int kGBytes = MS * kGRow, kXBytes = MS * kXRow;
  static constexpr int kStage = kGBytes * (HILO ? 2 : 1) + kXBytes;
  static constexpr int kGVec = MS * (BN / 8) / T, kXVec = MS * (BK / 16) / T;  // 16-byte pieces per thread
  static constexpr int kGStep = T / (BN / 8), kXStep = T / (BK / 16);          // rows between them
  static constexpr int kLds = 2 * KS * kStage;
  static_assert(WN == 64 && (FK == 8 || FK == 4), "the swizzles below assume these");
  static_assert(kGStep % 16 == 0 && kXStep % 16 == 0, "a thread's pieces share one swizzle");
  static_assert(KS == 1 || BN * BK * 4 <= kLds, "the second group's sums fit the stages");
};

// Rows of an LDS tile start on the same bank, so the pieces of a row are permuted
// by its number. A 16-bit transpose read takes units of 32 bytes of the rows r,
// r + 8, r + 16, r + 24 for four r at a time, an 8-bit one units of 16 bytes of 32
// rows: with these permutations each half of a read covers 256 bytes of banks once.
__device__ __forceinline__ int g_swizzle(int row) { return (row & 3) | ((row >> 1) & 4); }
template <int BK>
__device__ __forceinline__ int x_swizzle(int row) {
  return BK == 256 ? row & 15 : (row >> 1) & 7;
}

// Eight codes as operand values of the form, and its matrix instruction.
template <int XF, bool HILO>
__device__ __forceinline__ wg_i4 decode8(wg_i2 c) {
  if constexpr (HILO) return __builtin_bit_cast(wg_i4, f16x8<XF>((uint32_t)c[0], (uint32_t)c[1]));
  bf2v v[4];
  if constexpr (XF == kE4M3) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], 1.0f, false);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], 1.0f, true);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], 1.0f, false);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], 1.0f, true);
  } else {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[0], 1.0f, false);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[0], 1.0f, true);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[1], 1.0f, false);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[1], 1.0f, true);
  }
  return __builtin_bit_cast(wg_i4, wg_b8{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]});
}
template <bool HILO>
__device__ __forceinline__ v4f wg_mfma(wg_i4 x, wg_i4 g, v4f acc) {
  if constexpr (HILO)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, x), __builtin_bit_cast(h8v, g), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(wg_b8, x), __builtin_bit_cast(wg_b8, g), acc, 0, 0, 0);
}

// Largest finite |g * scale| of the 8 columns of a vector, as float32 bits, into m.
__device__ __forceinline__ void max8(const uint4& g, float scale, uint32_t* m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(vec_elem<kBF16>(g, e) * scale) & 0x7fffffffu;
    m[e] = max(m[e], b < kInfBits ? b : 0u);
  }
}
// The power of two that takes values up to m below 2^15.
__device__ __forceinline__ int f16_exponent(uint32_t m) { return m ? 141 - (int)(m >> 23) : 0; }

// Largest finite |g * scale| per column over one of gridDim.y runs of tokens: 512
// columns per workgroup, a wavefront per token.
__global__ __launch_bounds__(1024) void wgrad_colmax_kernel(WgradArgs a, int rows_per_part, uint32_t* out) {
  __shared__ uint32_t s[16][64][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (blockIdx.x * 64 + lane) * 8;
  const int m1 = min(a.m, (int)(blockIdx.y + 1) * rows_per_part);
  uint32_t m[8] = {};
  if (c < a.n) {
#pragma unroll 8
    for (int r = blockIdx.y * rows_per_part + wave; r < m1; r += 16)
      max8(*reinterpret_cast<const uint4*>(a.g + (size_t)r * a.n + c), a.x_scale[a.x_scale_per_row ? r : 0], m);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s[wave][lane][e] = m[e];
  __syncthreads();
  if (threadIdx.x >= 512) return;
  const int l = threadIdx.x >> 3, e = threadIdx.x & 7;
  uint32_t v = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) v = max(v, s[w][l][e]);
  const int col = (blockIdx.x * 64 + l) * 8 + e;
  if (col < a.n) out[(size_t)blockIdx.y * a.n + col] = v;
}

// Large shapes are bound by the matrix cores: 4096^3 bf16 118 to 124 us (1.11 to 1.16
// PFLOP/s; a large bf16 library product reaches 1.33), 8192 x 4096 x 4096 float32 446 to
// 496 us over several cards, two products per term. 2048 x 4096 x 1024 bf16, one
// 128 x 128 tile per CU, takes 22.6 to 26 us (0.66 to 0.76 PFLOP/s; the library's product
// of the decoded operands 28.0): 7 us that do not depend on the tokens and 9.0 to 9.5 per
// 1024 tokens. Counters there: matrix cores busy 29 %, vector instructions in 42 % of
// the issue slots (most of them the scaling of G), no LDS bank conflicts, and the same
// time with the operands in the caches: no unit is saturated, and what a step waits for
// is not known.
//
// Steps [step0, step1) of MS tokens; `part` selects the partial-sum slab when the
// tokens are split over workgroups.
// PER: the scale is read with each piece of G. The two-number form does so for one scale,
// too, with a step of zero; the one-number form has an instance of its own for it.
template <int XF, int BN, int BK, int KS, int MS, bool HILO, bool PER>
__global__ __launch_bounds__(512) void wgrad_kernel(WgradArgs a, int tiles_n, int tiles_k, int steps_per_part,
                                                    float* partials) {
  using C = WgCfg<BN, BK, KS, MS, HILO>;
  static_assert(PER || !HILO, "two numbers read the scale with each piece");
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  int tn, tk;
  tile_coords(xcd_remap(blockIdx.x, tiles_n * tiles_k), tiles_n, tiles_k, &tn, &tk);
  const int n0 = tn * BN, k0 = tk * BK;
  const int ks = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / C::T);
  const int t = threadIdx.x - ks * C::T;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wn = wave / C::kKW, wk = wave % C::kKW;
  const int nsteps_all = (int)(((int64_t)a.m + MS - 1) / MS);
  const int s_begin = blockIdx.y * steps_per_part;
  const int s_end = min(nsteps_all, s_begin + steps_per_part);

  // staging: piece v of a thread is row v * step + row0, one 16-byte chunk
  const int g_c = t % (BN / 8), g_r = t / (BN / 8);
  const int x_c = t % (BK / 16), x_r = t / (BK / 16);
  const int g_vo = n0 + g_c * 8 < a.n ? (int)((uint32_t)g_r * (uint32_t)a.n * 2u + (uint32_t)g_c * 16u) : kBadOffset;
  const int x_vo = k0 + x_c * 16 < a.k ? (int)((uint32_t)x_r * (uint32_t)a.k + (uint32_t)x_c * 16u) : kBadOffset;
  const int g_dst = g_r * C::kGRow + (((g_c >> 1) ^ g_swizzle(g_r)) << 5) + ((g_c & 1) << 4);
  const int x_dst = x_r * C::kXRow + ((x_c ^ x_swizzle<BK>(x_r)) << 4);
  const __amdgpu_buffer_rsrc_t s_rsrc = row_rsrc(a.x_scale, a.x_scale_per_row ? (uint32_t)a.m * 4u : 4u);
  const int s_step = a.x_scale_per_row ? 4 : 0;  // bytes from a token's scale to the next one's
  constexpr int H = HILO ? 2 : 1;

  // One scale for all tokens: its power of two is folded into G, which is exact, and the
  // sums are multiplied by the rest, in [1, 2) (the power of two keeps the sums in the
  // result's range). A scale that is zero, subnormal or not finite goes to the sums whole.
  float fold = 1.0f, rest = 1.0f;
  if (!PER && a.m > 0) {
    const uint32_t b = __float_as_uint(a.x_scale[0]), p2 = b & kInfBits;
    const bool normal = p2 != 0u && p2 != kInfBits;
    fold = __uint_as_float(normal ? p2 : 0x3f800000u);
    rest = __uint_as_float(normal ? (b & ~kInfBits) | 0x3f800000u : b);
  }

  // Two numbers: the exponents of the tile's columns, from the maxima that a pass
  // before this one wrote, or from the tile's own columns.
  __shared__ __attribute__((aligned(16))) int s_exp[HILO ? BN : 4];
  if constexpr (HILO) {
    uint32_t* s_max = reinterpret_cast<uint32_t*>(lds);
    constexpr int kRowsAt = C::kThreads / (BN / 8);
    static_assert(kRowsAt * BN * 4 <= C::kLds, "the columns' maxima fit the stages");
    if (!a.colmax) {
      const int c = threadIdx.x % (BN / 8), r0 = threadIdx.x / (BN / 8);
      uint32_t m[8] = {};
      if (n0 + c * 8 < a.n) {
        const int m1 = min(a.m, s_end * MS);
#pragma unroll 16
        for (int r = s_begin * MS + r0; r < m1; r += kRowsAt)
          max8(*reinterpret_cast<const uint4*>(a.g + (size_t)r * a.n + n0 + c * 8), a.x_scale[a.x_scale_per_row ? r : 0], m);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s_max[r0 * BN + c * 8 + e] = m[e];
      __syncthreads();
    }
    if (threadIdx.x < BN) {
      uint32_t m = 0;
      if (!a.colmax) {
#pragma unroll
        for (int r = 0; r < kRowsAt; ++r) m = max(m, s_max[r * BN + threadIdx.x]);
      } else if (n0 + (int)threadIdx.x < a.n) {
#pragma unroll 8
        for (int r = 0; r < a.colmax_parts; ++r) m = max(m, a.colmax[(size_t)r * a.n + n0 + threadIdx.x]);
      }
      s_exp[threadIdx.x] = f16_exponent(m);
    }
    __syncthreads();
  }

  // Operand reads. The swizzle only touches address bits below the row, and a
  // fragment's number only bits of the unit, so a fragment's address is the
  // lane's base with those bits flipped; rows and sub-steps are constant offsets.
  const int l16 = lane & 15, grp = lane >> 4;
  const int g_row = 8 * grp + (l16 >> 2);
  const int g_rd = g_row * C::kGRow + (((wn * C::FN) ^ g_swizzle(g_row)) << 5) + ((l16 & 3) << 3);
  const int x_row = 8 * grp + (l16 >> 1);
  const int x_rd = x_row * C::kXRow + (((wk * C::FK) ^ x_swizzle<BK>(x_row)) << 4) + ((l16 & 1) << 3);
  uint8_t* const lds_g = lds + ks * 2 * C::kStage;
  constexpr int kXOff = C::kGBytes * H;  // X after G in a stage

  // Loads: step s as range-checked buffers whose rows past m, and columns past n
  // and k, read zero. Piece v of G comes with its token's scale.
  uint4 rg[C::kGVec], rx[C::kXVec];
  float rs[C::kGVec];
  __amdgpu_buffer_rsrc_t g_rsrc, x_rsrc;
  int s_vo;  // byte offset of the scale of the thread's first row; past the extent where the step has no rows
  // The group's next step: first token (past the end it only advances) and the
  // tokens from there to the part's end.
  int next_m = (s_begin + ks) * MS;
  int next_left = min(a.m, s_end * MS) - next_m;
  const uint32_t n2 = (uint32_t)a.n * 2u, uk = (uint32_t)a.k;
  const uint8_t* next_g = reinterpret_cast<const uint8_t*>(a.g + (size_t)next_m * a.n + n0);
  const uint8_t* next_x = a.xq + (size_t)next_m * a.k + k0;
  const size_t g_adv = (size_t)KS * MS * n2, x_adv = (size_t)KS * MS * uk;
  auto set_step = [&]() {
    const bool any = next_left > 0;
    const uint32_t rows = (uint32_t)min(next_left, MS);
    g_rsrc = row_rsrc(next_g, any ? rows * n2 - (uint32_t)n0 * 2u : 0u);
    x_rsrc = row_rsrc(next_x, any ? rows * uk - (uint32_t)k0 : 0u);
    s_vo = any ? (next_m + g_r) * s_step : kBadOffset;
    next_g += g_adv;
    next_x += x_adv;
    next_m += KS * MS;
    next_left -= KS * MS;
  };
  auto load_g = [&](int v) {
    rg[v] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(g_rsrc, g_vo, (int)((uint32_t)(v * C::kGStep) * (uint32_t)a.n * 2u), 0));
    if constexpr (PER)
      rs[v] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(s_rsrc, s_vo, v * C::kGStep * s_step, 0));
  };
  auto load_x = [&](int v) {
    rx[v] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(x_rsrc, x_vo, (int)((uint32_t)(v * C::kXStep) * (uint32_t)a.k), 0));
  };
  auto store_g = [&](uint8_t* stage, int v) {
    uint32_t hi[4], lo[4];
    const float sc = PER ? rs[v] : fold;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f2v p = {vec_elem<kBF16>(rg[v], 2 * e) * sc, vec_elem<kBF16>(rg[v], 2 * e + 1) * sc};
      if constexpr (HILO) {
        const int* ex = s_exp + g_c * 8 + 2 * e;  // read at each use: registers are short
        p = f2v{__builtin_ldexpf(p[0], ex[0]), __builtin_ldexpf(p[1], ex[1])};
        const h2v h = __builtin_convertvector(p, h2v);
        hi[e] = __builtin_bit_cast(uint32_t, h);
        // v - hi in one instruction with hi as f16 (exact). It is at most 8; the clamp turns the NaN that an infinite or NaN hi
        // leaves into a finite lo, which adds nothing to it
        f2v q;
        asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(q[0]) : "v"(hi[e]), "v"(p[0]));
        asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(q[1]) : "v"(hi[e]), "v"(p[1]));
        q = f2v{__builtin_amdgcn_fmed3f(q[0], -8.0f, 8.0f), __builtin_amdgcn_fmed3f(q[1], -8.0f, 8.0f)};
        const h2v l = __builtin_convertvector(q, h2v);
        lo[e] = __builtin_bit_cast(uint32_t, l);
      } else {
        hi[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf2v));
      }
    }
    *reinterpret_cast<uint4*>(stage + g_dst + v * C::kGStep * C::kGRow) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (HILO)
      *reinterpret_cast<uint4*>(stage + C::kGBytes + g_dst + v * C::kGStep * C::kGRow) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  };
  auto store_x = [&](uint8_t* stage, int v) {
    *reinterpret_cast<uint4*>(stage + kXOff + x_dst + v * C::kXStep * C::kXRow) = rx[v];
  };

  v4f acc[C::FK][C::FN];
#pragma unroll
  for (int i = 0; i < C::FK; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  auto read_g = [&](const uint8_t* stage, int ss, wg_i4 (&f)[H][C::FN]) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const wg_s4 a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (HQ_LDS wg_s4*)(stage + h * C::kGBytes + (g_rd ^ (j << 5)) + ss * 32 * C::kGRow));
        const wg_s4 a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (HQ_LDS wg_s4*)(stage + h * C::kGBytes + (g_rd ^ (j << 5)) + (ss * 32 + 4) * C::kGRow));
        f[h][j] = __builtin_bit_cast(wg_i4, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
      }
  };
  auto read_x = [&](const uint8_t* stage, int slot) -> wg_i2 {
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (HQ_LDS wg_i2*)(stage + kXOff + (x_rd ^ ((slot % C::FK) << 4)) + (slot / C::FK) * 32 * C::kXRow));
  };

  // One step of MS tokens as slots of one X fragment each. A slot reads the X
  // fragment of two slots ahead, converts the next slot's, runs its own MFMAs and
  // takes its share of the staging: a piece of the next step is converted, stored
  // to the other stage and replaced by its load for the step after. The pieces
  // are all stored two slots before the step ends; the barrier stands there, by
  // which time every read of this stage has been issued too, and the last two slots
  // read the next stage's first fragments (with one sub-step per step, G's after the
  // last MFMAs). So no MFMA waits for X at a step's start, and the VALU work lies
  // between matrix instructions (the group barriers ask for that order).
  constexpr int kSub = MS / 32, kSlots = kSub * C::FK, kPieces = C::kGVec + C::kXVec, kFill = kSlots - 2;
  static_assert(kSlots % 2 == 0 && kFill >= 2, "slots");
  wg_i4 fg[2][H][C::FN];
  wg_i2 raw[2];
  wg_i4 xb[2];
  auto step = [&](int buf) {
    const uint8_t* cur = lds_g + buf * C::kStage;
    uint8_t* nxt = lds_g + (buf ^ 1) * C::kStage;
#pragma unroll
    for (int sl = 0; sl < kSlots; ++sl) {
      const int ss = sl / C::FK, i = sl % C::FK;
      raw[sl & 1] = sl + 2 < kSlots ? read_x(cur, sl + 2) : read_x(nxt, sl + 2 - kSlots);
      if (i == C::FK / 2 - 1 && ss + 1 < kSub) read_g(cur, ss + 1, fg[(ss + 1) & 1]);
      if (kSub % 2 == 0 && sl == kFill) read_g(nxt, 0, fg[0]);
      xb[(sl + 1) & 1] = decode8<XF, HILO>(raw[(sl + 1) & 1]);
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
          acc[i][j] = wg_mfma<HILO>(xb[sl & 1], fg[ss & 1][h][j], acc[i][j]);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        if (p * kFill / kPieces != sl) continue;
        if (p < C::kGVec) {
          store_g(nxt, p);
          load_g(p);
        } else {
          store_x(nxt, p - C::kGVec);
          load_x(p - C::kGVec);
        }
      }
#pragma unroll
      for (int q = 0; q < H * C::FN; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one matrix instruction,
        __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);  // then vector ones
      }
      __builtin_amdgcn_sched_barrier(0);
      if (kSub % 2 == 1 && sl == kSlots - 1) read_g(nxt, 0, fg[0]);
      if (sl == kFill - 1) __syncthreads();
    }
  };

  // Step s is loaded two steps ahead into registers and stored one step ahead;
  // both groups of KS == 2 pass the same number of barriers (steps past the end
  // hold zeros).
  const int iters = (max(s_end - s_begin, 0) + KS - 1) / KS;
  auto load_all = [&]() {
    set_step();
#pragma unroll
    for (int v = 0; v < C::kGVec; ++v) load_g(v);
#pragma unroll
    for (int v = 0; v < C::kXVec; ++v) load_x(v);
  };
  load_all();
#pragma unroll
  for (int v = 0; v < C::kGVec; ++v) store_g(lds_g, v);
#pragma unroll
  for (int v = 0; v < C::kXVec; ++v) store_x(lds_g, v);
  load_all();
  __syncthreads();
  read_g(lds_g, 0, fg[0]);
  raw[0] = read_x(lds_g, 0);
  raw[1] = read_x(lds_g, 1);
  xb[0] = decode8<XF, HILO>(raw[0]);
  if constexpr (kSub % 2 == 0 && PER) {
    // two steps per iteration: the stages' offsets are constants
    for (int i = 0; i < iters; i += 2) {
      set_step();
      step(0);
      if (i + 1 == iters) break;
      set_step();
      step(1);
    }
  } else {
    // one. With one sub-step its fragments of G are read after the step before's last MFMAs
    // (reading them earlier into registers of their own took 256 registers and spilled);
    // with one scale for all tokens the product of the sums with it left the two-step
    // loop's 256 x 256 tile 168 registers short (845 us at 4096^3)
    for (int i = 0; i < iters; ++i) {
      set_step();
      step(i & 1);
    }
  }
  __syncthreads();

  if constexpr (KS == 2) {
    v4f* part = reinterpret_cast<v4f*>(lds);
    if (ks == 1) {
#pragma unroll
      for (int i = 0; i < C::FK; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) part[(i * C::FN + j) * C::T + t] = acc[i][j];
    }
    __syncthreads();
    if (ks == 1) return;
#pragma unroll
    for (int i = 0; i < C::FK; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] += part[(i * C::FN + j) * C::T + t];
  }

  // Lane l of fragment (i, j) holds columns k = 16 i + 4 (l / 16) .. +3 of row
  // n = 16 j + l % 16 of its wavefront's block.
#pragma unroll
  for (int j = 0; j < C::FN; ++j) {
    const int n = n0 + wn * C::WN + j * 16 + l16;
    if (n >= a.n) continue;
    const int back = HILO ? -s_exp[wn * C::WN + j * 16 + l16] : 0;
#pragma unroll
    for (int i = 0; i < C::FK; ++i) {
      const int k = k0 + wk * C::WK + i * 16 + 4 * grp;
      if (k >= a.k) continue;
      const size_t at = (size_t)n * a.k + k;
      v4f v = acc[i][j];
      if constexpr (HILO) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_ldexpf(v[e], back);
      }
      if constexpr (!PER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= rest;
      }
      if (partials) {
        *reinterpret_cast<v4f*>(partials + (size_t)blockIdx.y * a.n * a.k + at) = v;
        continue;
      }
      if (a.base) v += *reinterpret_cast<const v4f*>(a.base + at);
      if (HILO && a.out_f32) {
        *reinterpret_cast<v4f*>(static_cast<float*>(a.dw) + at) = v;
      } else {
        const bf2v b0 = __builtin_convertvector((f2v{v[0], v[1]}), bf2v), b1 = __builtin_convertvector((f2v{v[2], v[3]}), bf2v);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dw) + at) =
            make_uint2(__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1));
      }
    }
  }
}

// The split form's sums, added in the order of the tokens.
__global__ __launch_bounds__(256) void wgrad_sum_kernel(const float* __restrict__ partials, int parts, size_t nvec,
                                                        const float* base, void* dw, int out_f32) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= nvec) return;
  v4f v = reinterpret_cast<const v4f*>(partials)[i];
  for (int p = 1; p < parts; ++p) v += reinterpret_cast<const v4f*>(partials)[(size_t)p * nvec + i];
  if (base) v += reinterpret_cast<const v4f*>(base)[i];
  if (out_f32) {
    static_cast<v4f*>(dw)[i] = v;
  } else {
    const bf2v b0 = __builtin_convertvector((f2v{v[0], v[1]}), bf2v), b1 = __builtin_convertvector((f2v{v[2], v[3]}), bf2v);
    static_cast<uint2*>(dw)[i] = make_uint2(__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1));
  }
}

// Up to this many tokens a bf16 result, too, takes the two-number form: the call's
// time is that of writing dW.
constexpr int kWgTwoNumbersM = 64;
// Up to this many tokens a workgroup of that form finds its columns' maxima itself,
// a few reads; beyond, a pass of its own reads G once for all.
constexpr int kWgOwnMaxM = 512;

// Launch plan: the 256 x 256 tile where its tiles fill the CUs, else 128 x 128;
// where those leave CUs idle too and there are many tokens, the tokens are split.
// Workspace: the columns' maxima [max_parts, n], then the partial sums [parts, n, k].
struct WgPlan {
  bool hilo, big;
  int tiles_n, tiles_k, steps, parts, max_parts;
  size_t max_bytes, bytes;
};
static WgPlan wgrad_plan(int m, int n, int k, bool two_numbers) {
  WgPlan p{};
  p.hilo = two_numbers || m <= kWgTwoNumbersM;
  const int ms = p.hilo ? 32 : 64;
  auto tiles = [&](int b) { return (int64_t)((n + b - 1) / b) * ((k + b - 1) / b); };
  p.big = tiles(256) >= kNumCUs * 3 / 4;
  const int b = p.big ? 256 : 128;
  p.tiles_n = (n + b - 1) / b;
  p.tiles_k = (k + b - 1) / b;
  const int nsteps = (int)(((int64_t)m + ms - 1) / ms);
  p.parts = 1;
  while (!p.big && tiles(b) * p.parts * 2 <= kNumCUs && nsteps >= p.parts * 2 * 8) p.parts *= 2;
  p.steps = (nsteps + p.parts - 1) / p.parts;
  if (p.hilo && m > kWgOwnMaxM) {
    const int xb = (n + 511) / 512;
    p.max_parts = xb >= kNumCUs ? 1 : kNumCUs / xb < 32 ? kNumCUs / xb : 32;
  }
  p.max_bytes = (size_t)p.max_parts * n * 4;
  p.bytes = p.max_bytes + (p.parts > 1 ? (size_t)p.parts * n * k * 4 : 0);
  return p;
}

size_t wgrad_workspace_bytes(int m, int n, int k, bool two_numbers) { return wgrad_plan(m, n, k, two_numbers).bytes; }

template <int XF, bool HILO, bool PER>
static hipError_t launch_wgrad_t(WgradArgs a, WgPlan p, uint8_t* workspace, size_t workspace_bytes, hipStream_t st) {
  constexpr int MS = HILO ? 32 : 64;
  float* partials = nullptr;
  if (p.parts > 1 && workspace_bytes >= p.bytes) {
    partials = reinterpret_cast<float*>(workspace + p.max_bytes);
  } else {
    p.steps *= p.parts;
    p.parts = 1;
  }
  if (p.max_parts > 0 && workspace_bytes >= p.max_bytes) {
    uint32_t* out = reinterpret_cast<uint32_t*>(workspace);
    hipLaunchKernelGGL(wgrad_colmax_kernel, dim3((a.n + 511) / 512, p.max_parts), dim3(1024), 0, st, a,
                       (a.m + p.max_parts - 1) / p.max_parts, out);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.colmax = out;
    a.colmax_parts = p.max_parts;
  }
  const dim3 grid(p.tiles_n * p.tiles_k, p.parts);
  if (p.big)
    hipLaunchKernelGGL((wgrad_kernel<XF, 256, 256, 1, MS, HILO, PER>), grid, dim3(512), 0, st, a, p.tiles_n, p.tiles_k, p.steps,
                       partials);
  else
    hipLaunchKernelGGL((wgrad_kernel<XF, 128, 128, 2, MS, HILO, PER>), grid, dim3(512), 0, st, a, p.tiles_n, p.tiles_k, p.steps,
                       partials);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !partials) return e;
  const size_t nvec = (size_t)a.n * a.k / 4;
  hipLaunchKernelGGL(wgrad_sum_kernel, dim3((unsigned)((nvec + 255) / 256)), dim3(256), 0, st, partials, p.parts, nvec, a.base,
                     a.dw, a.out_f32);
  return hipGetLastError();
}

template <int XF>
static hipError_t launch_wgrad_x(const WgradArgs& a, const WgPlan& p, uint8_t* workspace, size_t workspace_bytes, hipStream_t st) {
  if (p.hilo) return launch_wgrad_t<XF, true, true>(a, p, workspace, workspace_bytes, st);
  return a.x_scale_per_row ? launch_wgrad_t<XF, false, true>(a, p, workspace, workspace_bytes, st)
                           : launch_wgrad_t<XF, false, false>(a, p, workspace, workspace_bytes, st);
}

hipError_t launch_wgrad(const WgradArgs& a, int xf, void* workspace, size_t workspace_bytes, hipStream_t st) {
  const WgPlan p = wgrad_plan(a.m, a.n, a.k, a.out_f32 || a.strict);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return xf == kE4M3 ? launch_wgrad_x<kE4M3>(a, p, ws, workspace_bytes, st)
                     : launch_wgrad_x<kE5M2>(a, p, ws, workspace_bytes, st);
}

}  // namespace hq
