// The mixture-of-experts layer of a decode step and its router, gfx950.
//
//   route     ids = the topk largest logits of a token, weights = their scores
//             (softmax over all experts or logistic), renormalised or not
//   layer     for a token t and its j-th expert e:
//             z[t,j] = x_scale[t] w1_scale[e] (dec(XQ[t]) . dec(W1[e])) + b1[e]
//             a[t,j] = act(z)  or  act(z[:F]) * z[F:]
//             out[t] = sum_j weights[t,j] (w2_scale[e] (a[t,j] . dec(W2[e])) + b2[e]) + residual[t]
#include "gemm_kernels.h"
#include "hq_row.h"

namespace hq {

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------
// A token belongs to G lanes (16, so that its maxima need only lane moves within a
// row of lanes, or 64) that hold V of its logits each: lane l has experts l, l + G,
// ... The k-th largest is found k times over: the lanes' maxima, then the lowest
// index that holds the maximum, which leaves the race. All in registers: one read of
// the logits.
constexpr int kMaxTopk = 16;

template <int G, class F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // swap neighbours
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // swap pairs
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // half-row mirror
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // row mirror
  if constexpr (G == 64) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return __uint_as_float(group_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ int group_min(int v) {
  return (int)group_reduce<G>((uint32_t)v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

// A logit; NaN counts as -Inf.
template <int XT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  const float v = XT == kF32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  return v == v ? v : -__builtin_inff();
}
// exp(l - m) for l <= m; equal infinities differ by nothing.
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }
// log of the logistic function, and 1 / (1 + exp(-l)).
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// The renormalised weights of the slots that lanes 0 .. of a group hold (`in`: this
// lane holds one): scores divided by their sum, from the scores' logarithms, so that
// logits far below 0 do not underflow.
template <int G>
__device__ __forceinline__ float renormalised(float l, bool in, int score) {
  const float s = !in ? -__builtin_inff() : score == kRouteSigmoid ? log_sigmoid(l) : l;
  const float top = group_max<G>(s);  // by all lanes of the group, also those without a slot
  const float e = in ? exp_below(s, top) : 0.0f;
  const float total = group_sum<G>(e);
  return in ? e / total : 0.0f;
}

template <int XT, int G, int V>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  constexpr int kRows = 256 / G;  // tokens per workgroup
  const int l = threadIdx.x % G;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G; row < a.tokens; row += (int64_t)gridDim.x * kRows) {
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = l + G * j;
      v[j] = e < a.experts ? load_logit<XT>(a.logits, row * a.experts + e) : -__builtin_inff();
    }
    float top = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) top = fmaxf(top, v[j]);
    top = group_max<G>(top);
    float all = 0.0f;  // sum of the exponentials of all experts
    if (a.score == kRouteSoftmax && !a.renormalize) {
#pragma unroll
      for (int j = 0; j < V; ++j) all += v[j] == -__builtin_inff() ? 0.0f : exp_below(v[j], top);
      all = group_sum<G>(all);
    }
    // slot r stays with lane r
    int id = -1;
    float mine = 0.0f, m = top;
    for (int r = 0; r < a.topk; ++r) {
      int at = 0x7fffffff;
#pragma unroll
      for (int j = V - 1; j >= 0; --j) at = v[j] == m ? l + G * j : at;
      at = group_min<G>(at);
      const bool found = m != -__builtin_inff();
      if (l == r && found) {
        id = at;
        mine = m;
      }
      m = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (found && at == l + G * j) v[j] = -__builtin_inff();
        m = fmaxf(m, v[j]);
      }
      m = group_max<G>(m);
    }
    float w = 0.0f;
    if (a.renormalize) w = renormalised<G>(mine, id >= 0, a.score);
    else if (id >= 0) w = a.score == kRouteSigmoid ? sigmoid(mine) : exp_below(mine, top) / all;
    if (l < a.topk) {
      a.ids[row * a.topk + l] = id;
      a.weights[row * a.topk + l] = w;
    }
  }
}

// Backward pass, from the logits and the chosen ids (with the score p, the weight W
// and its gradient g of a slot):
//   renormalised softmax    dl = W (g - sum_slots g W)
//   renormalised logistic   dl = W (g - sum_slots g W) (1 - p)
//   logistic                dl = g p (1 - p)
//   softmax                 dl_e = p_e (sum of e's slots g - sum_slots g p), every expert
template <int XT, int G, int V>
__global__ __launch_bounds__(256) void moe_route_bwd_kernel(RouteBwdArgs a) {
  constexpr int kRows = 256 / G;
  const int l = threadIdx.x % G;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G; row < a.tokens; row += (int64_t)gridDim.x * kRows) {
    // lane r holds slot r
    int id = l < a.topk ? a.ids[row * a.topk + l] : -1;
    const bool in = id >= 0 && id < a.experts;
    if (!in) id = -1;
    float g = in ? a.dweights[row * a.topk + l] : 0.0f;
    const bool full = a.score == kRouteSoftmax && !a.renormalize;
    if (!full) {
      const float mine = in ? load_logit<XT>(a.logits, row * a.experts + id) : 0.0f;
      if (a.renormalize) {
        const float w = renormalised<G>(mine, in, a.score);
        const float dot = group_sum<G>(g * w);
        g = in ? w * (g - dot) : 0.0f;
        if (a.score == kRouteSigmoid) g *= sigmoid(-mine);
      } else {
        g *= sigmoid(mine) * sigmoid(-mine);
      }
    }
    float acc[V], p[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = p[j] = 0.0f;
    for (int r = 0; r < a.topk; ++r) {
      const int e = __shfl(id, r, G);
      const float s = __shfl(g, r, G);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += e == l + G * j ? s : 0.0f;
    }
    if (full) {
      float top = -__builtin_inff(), all = 0.0f, dot = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = l + G * j;
        p[j] = e < a.experts ? load_logit<XT>(a.logits, row * a.experts + e) : -__builtin_inff();
        top = fmaxf(top, p[j]);
      }
      top = group_max<G>(top);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        p[j] = p[j] == -__builtin_inff() ? 0.0f : exp_below(p[j], top);
        all += p[j];
      }
      all = group_sum<G>(all);
      const float inv = all > 0.0f ? 1.0f / all : 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        p[j] *= inv;
        dot = fmaf(acc[j], p[j], dot);
      }
      dot = group_sum<G>(dot);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = p[j] * (acc[j] - dot);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = l + G * j;
      if (e >= a.experts) continue;
      if constexpr (XT == kF32) static_cast<float*>(a.dlogits)[row * a.experts + e] = acc[j];
      else static_cast<uint16_t*>(a.dlogits)[row * a.experts + e] = (uint16_t)f32_to_bf16_rne(acc[j]);
    }
  }
}

constexpr int64_t kMaxRouteBlocks = 1 << 20;

#define HQ_ROUTE(KERNEL, XT, G, V)                                                                                      \
  do {                                                                                                                  \
    const int64_t want = ((int64_t)a.tokens + 256 / G - 1) / (256 / G);                                                 \
    hipLaunchKernelGGL((KERNEL<XT, G, V>), dim3((unsigned)(want < kMaxRouteBlocks ? want : kMaxRouteBlocks)), dim3(256), \
                       0, st, a);                                                                                       \
    return hipGetLastError();                                                                                           \
  } while (0)
#define HQ_ROUTE_X(KERNEL, XT)                           \
  do {                                                   \
    if (a.experts <= 64) HQ_ROUTE(KERNEL, XT, 16, 4);    \
    if (a.experts <= 128) HQ_ROUTE(KERNEL, XT, 16, 8);   \
    if (a.experts <= 256) HQ_ROUTE(KERNEL, XT, 16, 16);  \
    if (a.experts <= 512) HQ_ROUTE(KERNEL, XT, 64, 8);   \
    HQ_ROUTE(KERNEL, XT, 64, 16);                        \
  } while (0)

hipError_t launch_moe_route(const RouteArgs& a, int xt, hipStream_t st) {
  if (xt == kBF16) HQ_ROUTE_X(moe_route_kernel, kBF16);
  HQ_ROUTE_X(moe_route_kernel, kF32);
}
hipError_t launch_moe_route_bwd(const RouteBwdArgs& a, int xt, hipStream_t st) {
  if (xt == kBF16) HQ_ROUTE_X(moe_route_bwd_kernel, kBF16);
  HQ_ROUTE_X(moe_route_bwd_kernel, kF32);
}
#undef HQ_ROUTE_X
#undef HQ_ROUTE

// ---------------------------------------------------------------------------
// the layer: which experts, which rows
// ---------------------------------------------------------------------------
// A step of at most 64 tokens: one lane per token finds an expert's rows, and the
// experts that are asked for are a bitmap in LDS. Every wavefront does both by itself.
constexpr int kMoeMaxTokens = 64, kMoeMaxPairs = kMoeMaxTokens * kMaxTopk, kMoeMaxExperts = 1024;

struct MoeLds {
  int ids[kMoeMaxPairs];
  float weights[kMoeMaxPairs];
  uint32_t bits[kMoeMaxExperts / 32];
};

// Fills s; ends with a barrier.
template <int THREADS>
__device__ __forceinline__ void moe_load_pairs(const MoeArgs& a, MoeLds& s) {
  const int pairs = a.tokens * a.topk;
  if (threadIdx.x < kMoeMaxExperts / 32) s.bits[threadIdx.x] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += THREADS) {
    const int e = a.ids[p];
    s.ids[p] = e;
    s.weights[p] = a.weights[p];
    if ((unsigned)e < (unsigned)a.experts) atomicOr(&s.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// The experts that are asked for, in order: lane i < 32 holds 32 of the bits and the
// number of bits before them.
struct ActiveExperts {
  uint32_t word;
  int before, count;
  __device__ explicit ActiveExperts(const MoeLds& s) {
    const int lane = threadIdx.x & 63;
    word = lane < 32 ? s.bits[lane] : 0u;
    int upto = __popc(word);
    const int own = upto;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    before = upto - own;
    count = __builtin_amdgcn_readlane(upto, 63);
  }
  // The i-th of them, i < count.
  __device__ int at(int i) const {
    const uint64_t m = __ballot(before <= i && i < before + __popc(word));
    const int src = __builtin_ctzll(m);
    uint32_t w = __builtin_amdgcn_readlane(word, src);
    for (int k = i - __builtin_amdgcn_readlane(before, src); k > 0; --k) w &= w - 1;
    return src * 32 + __builtin_ctz(w);
  }
};

// The tokens that chose expert e, in order: their first pair with it, and the sum of
// their weights for it (a token that names an expert twice has one row). rows and
// wts have 64 entries of this wavefront's own.
__device__ __forceinline__ int moe_expert_rows(const MoeArgs& a, const MoeLds& s, int e, int* rows, float* wts) {
  const int t = threadIdx.x & 63;
  int p = -1;
  float w = 0.0f;
  if (t < a.tokens) {
    for (int j = 0; j < a.topk; ++j) {
      const int q = t * a.topk + j;
      if (s.ids[q] == e) {
        if (p < 0) p = q;
        w += s.weights[q];
      }
    }
  }
  const uint64_t m = __ballot(p >= 0);
  if (p >= 0) {
    const int at = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
    rows[at] = p;
    wts[at] = w;
  }
  // LDS operations of one wavefront complete in order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  return __popcll(m);
}

// ---------------------------------------------------------------------------
// first product and activation
// ---------------------------------------------------------------------------
constexpr int kMoeWaves = 8;

// A workgroup owns two weight fragments of one expert: 16 columns of the first half
// and the same columns of the second (gated), or 32 columns. Its wavefronts take the
// K blocks w, w + 8, ..., KPW of them at a time, and meet in LDS.
template <int XF, int WF, int MB, bool GATED>
__global__ __launch_bounds__(64 * kMoeWaves) void moe_up_kernel(MoeArgs a, int strips, int act) {
  constexpr int KPW = 2;
  __shared__ MoeLds s;
  __shared__ int s_rows[kMoeWaves][kMoeMaxTokens];
  __shared__ float s_wts[kMoeWaves][kMoeMaxTokens];
  __shared__ __attribute__((aligned(16))) v4f red[kMoeWaves][2 * MB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = blockIdx.x / strips, strip = blockIdx.x % strips;
  moe_load_pairs<64 * kMoeWaves>(a, s);
  const ActiveExperts active(s);
  if (slot >= active.count) return;
  const int e = active.at(slot);
  const int nrows = moe_expert_rows(a, s, e, s_rows[wave], s_wts[wave]);

  const int K = a.hidden, nkb = (K + kBK - 1) / kBK;
  const int n1 = GATED ? 2 * a.inner : a.inner;
  const int frag[2] = {GATED ? strip : 2 * strip, GATED ? a.inner / 16 + strip : 2 * strip + 1};
  const uint8_t* w = a.w1 + (size_t)e * (size_t)frag_rows(n1) * nkb * kFragBytes;
  __amdgpu_buffer_rsrc_t w_rsrc[2];
#pragma unroll
  for (int f = 0; f < 2; ++f)
    w_rsrc[f] = __builtin_amdgcn_make_buffer_rsrc((void*)(w + (size_t)frag[f] * nkb * kFragBytes), (short)0, nkb * kFragBytes,
                                                  kRsrcFlags);
  const __amdgpu_buffer_rsrc_t x_rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)a.xq, (short)0, a.tokens * K, kRsrcFlags);
  const int xr = lane & 15, xc = 32 * (lane >> 4);

  for (int r0 = 0; r0 < nrows; r0 += 16 * MB) {
    int xo[MB];  // byte offset of the lane's row
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int r = r0 + 16 * i + xr;
      xo[i] = r < nrows ? s_rows[wave][r] / a.topk * K : kBadOffset;
    }
    v4f acc[2][MB];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < MB; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb0 = wave; kb0 < nkb; kb0 += KPW * kMoeWaves) {
      uint4 fb[KPW][2][2], fx[KPW][MB][2];
#pragma unroll
      for (int j = 0; j < KPW; ++j) {
        const int kb = kb0 + j * kMoeWaves;
        const int wo = kb < nkb ? lane * 16 : kBadOffset;  // the scalar offset is not range-checked
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            fb[j][f][h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(w_rsrc[f], wo + h * 1024, min(kb, nkb - 1) * kFragBytes, kNtLoad));
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = kb * kBK + xc + 16 * h;
            fx[j][i][h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(x_rsrc, col < K && xo[i] >= 0 ? xo[i] + col : kBadOffset, 0, 0));
          }
      }
      __builtin_amdgcn_sched_barrier(0);  // every load of the chunk ahead of its first product
#pragma unroll
      for (int j = 0; j < KPW; ++j) {
        h8v wh[2][4];
#pragma unroll
        for (int f = 0; f < 2; ++f) f16_frag<WF>(fb[j][f][0], fb[j][f][1], wh[f]);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          h8v xh[4];
          f16_frag<XF>(fx[j][i][0], fx[j][i][1], xh);
#pragma unroll
          for (int f = 0; f < 2; ++f) acc[f][i] = mfma_f16x4(wh[f], xh, acc[f][i]);
        }
      }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < MB; ++i) red[wave][f * MB + i][lane] = acc[f][i];
    __syncthreads();
    // Wavefront i finishes the 16 rows i (gated), wavefront 2 i + f their fragment f.
    const int i = GATED ? wave : wave >> 1;
    const int r = r0 + 16 * i + xr;
    if (i < MB && r < nrows) {
      const int pair = s_rows[wave][r];
      const float xs = a.x_scale[a.x_scale_per_row ? pair / a.topk : 0];
      float z[2][4];
#pragma unroll
      for (int f = 0; f < (GATED ? 2 : 1); ++f) {
        const int ff = GATED ? f : wave & 1;
        v4f t = red[0][ff * MB + i][lane];
#pragma unroll
        for (int v = 1; v < kMoeWaves; ++v) t += red[v][ff * MB + i][lane];
        const int nb = ff ? frag[1] : frag[0];
        const int col = 32 * (nb >> 1) + 8 * (lane >> 4) + 4 * (nb & 1);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const size_t at = (size_t)e * n1 + min(col + q, n1 - 1);
          z[f][q] = t[q] * xs * a.s1[a.s1_per_col ? at : e];
          if (a.b1) z[f][q] += __uint_as_float((uint32_t)a.b1[at] << 16);
        }
      }
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[q] = z[0][q];
      }
      fused_act<4>(act, o);
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] *= z[1][q];
      }
      const int nb = GATED || !(wave & 1) ? frag[0] : frag[1];
      const int col = 32 * (nb >> 1) + 8 * (lane >> 4) + 4 * (nb & 1);
      if (col < a.inner) {
        const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{o[0], o[1]}), bf2v));
        const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{o[2], o[3]}), bf2v));
        *reinterpret_cast<uint2*>(a.a + (size_t)pair * a.inner + col) = make_uint2(w0, w1);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// second product and weighted sum
// ---------------------------------------------------------------------------
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
template <int FMT>
__device__ __forceinline__ b8v bf16x8(uint32_t d0, uint32_t d1) {
  bf2v a, b, c, d;
  if constexpr (FMT == kE4M3) {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, 1.0f, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, 1.0f, true);
  } else {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(d0, 1.0f, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(d0, 1.0f, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(d1, 1.0f, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(d1, 1.0f, true);
  }
  return b8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A workgroup owns FB weight fragments (16 FB output columns) of every expert, and all
// tokens; the (expert, K block) pairs are dealt in runs over its wavefronts and over
// `splits` workgroups. A wavefront adds an expert's weighted rows into sums of its own
// in LDS ([token][column], TB tokens), so no two lanes meet; at the end the wavefronts'
// sums are added in order, and with splits > 1 the last workgroup to arrive adds the
// workgroups' sums, in order too: the result does not depend on who ends first.
template <int WF, int MB, int FB, int TB>
__global__ __launch_bounds__(64 * kMoeWaves) void moe_down_kernel(MoeArgs a, int splits, uint32_t* counters, float* partials) {
  constexpr int KPW = 2;
  constexpr int kCols = 16 * FB, kPitch = kCols + 4;
  __shared__ MoeLds s;
  __shared__ int s_rows[kMoeWaves][kMoeMaxTokens];
  __shared__ float s_wts[kMoeWaves][kMoeMaxTokens];
  __shared__ __attribute__((aligned(16))) float sums[kMoeWaves][TB][kPitch];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strip = blockIdx.x / splits, split = blockIdx.x % splits;
  for (int i = lane; i < a.tokens * (kPitch / 4); i += 64)
    *reinterpret_cast<v4f*>(&sums[wave][0][0] + 4 * i) = v4f{0.f, 0.f, 0.f, 0.f};
  moe_load_pairs<64 * kMoeWaves>(a, s);
  const ActiveExperts active(s);

  const int K = a.inner, nkb = (K + kBK - 1) / kBK;
  const int nfrag = frag_rows(a.hidden);
  const int nb0 = strip * FB;
  const int xr = lane & 15, xq = lane >> 4;
  const __amdgpu_buffer_rsrc_t a_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)a.a, (short)0, a.tokens * a.topk * K * 2, kRsrcFlags);
  const int64_t items = (int64_t)active.count * nkb;
  const int runs = splits * kMoeWaves, run = split * kMoeWaves + wave;
  const int last = (int)(items * (run + 1) / runs);
  for (int it = (int)(items * run / runs); it < last;) {
    const int slot = it / nkb, kb0 = it % nkb, kb1 = min(nkb, kb0 + last - it);
    it += kb1 - kb0;
    const int e = active.at(slot);
    const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(a.w2 + ((size_t)e * nfrag + nb0) * nkb * kFragBytes), (short)0, FB * nkb * kFragBytes, kRsrcFlags);
    const int nrows = moe_expert_rows(a, s, e, s_rows[wave], s_wts[wave]);
    // the lane's 4 columns of each fragment: scales and, where the run holds the first K block, the bias
    float sc[FB][4], bias[FB][4];
#pragma unroll
    for (int f = 0; f < FB; ++f) {
      const int nb = nb0 + f;
      const int col = 32 * (nb >> 1) + 8 * xq + 4 * (nb & 1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const size_t at = (size_t)e * a.hidden + min(col + q, a.hidden - 1);
        sc[f][q] = a.s2[a.s2_per_col ? at : e];
        bias[f][q] = a.b2 && kb0 == 0 ? __uint_as_float((uint32_t)a.b2[at] << 16) : 0.0f;
      }
    }
    for (int r0 = 0; r0 < nrows; r0 += 16 * MB) {
      int ao[MB];  // byte offset of the lane's row
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int r = r0 + 16 * i + xr;
        ao[i] = r < nrows ? s_rows[wave][r] * K * 2 : kBadOffset;
      }
      v4f acc[FB][MB];
#pragma unroll
      for (int f = 0; f < FB; ++f)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
      for (int kc = kb0; kc < kb1; kc += KPW) {
        uint4 fb[KPW][FB][2], fa[KPW][MB][4];
#pragma unroll
        for (int j = 0; j < KPW; ++j) {
          const int kb = kc + j;
          const bool in = kb < kb1;
#pragma unroll
          for (int f = 0; f < FB; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              fb[j][f][h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(w_rsrc, in ? lane * 16 + h * 1024 : kBadOffset,
                                                                           (f * nkb + min(kb, nkb - 1)) * kFragBytes, kNtLoad));
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const int col = kb * kBK + 32 * xq + 8 * m;
              fa[j][i][m] = as_uint4(
                  __builtin_amdgcn_raw_buffer_load_b128(a_rsrc, in && col < K && ao[i] >= 0 ? ao[i] + 2 * col : kBadOffset, 0, 0));
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // every load of the chunk ahead of its first product
#pragma unroll
        for (int j = 0; j < KPW; ++j)
#pragma unroll
          for (int f = 0; f < FB; ++f) {
            const uint4 &lo = fb[j][f][0], &hi = fb[j][f][1];
            const b8v w[4] = {bf16x8<WF>(lo.x, lo.y), bf16x8<WF>(lo.z, lo.w), bf16x8<WF>(hi.x, hi.y), bf16x8<WF>(hi.z, hi.w)};
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
              for (int m = 0; m < 4; ++m)
                acc[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[m], __builtin_bit_cast(b8v, fa[j][i][m]), acc[f][i], 0, 0, 0);
          }
      }
      // lane l holds row l % 16 and 4 columns of each fragment
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int r = r0 + 16 * i + xr;
        if (r >= nrows) continue;
        float* row = sums[wave][s_rows[wave][r] / a.topk];
        const float wt = s_wts[wave][r];
#pragma unroll
        for (int f = 0; f < FB; ++f) {
          v4f* p = reinterpret_cast<v4f*>(row + 16 * f + 4 * xq);
          v4f t = *p;
#pragma unroll
          for (int q = 0; q < 4; ++q) t[q] = fmaf(wt, fmaf(acc[f][i][q], sc[f][q], bias[f][q]), t[q]);
          *p = t;
        }
      }
    }
  }
  __syncthreads();

  // 4 columns of a token per thread
  const int units = a.tokens * 4 * FB;
  auto column = [&](int u) {
    const int nb = nb0 + u % (4 * FB) / 4;
    return 32 * (nb >> 1) + 8 * (u % 4) + 4 * (nb & 1);
  };
  auto finish = [&](int u, v4f t) {
    const int col = column(u);
    if (col >= a.hidden) return;
    const size_t off = (size_t)(u / (4 * FB)) * a.hidden + col;
    if (a.residual) {
      const uint2 r = *reinterpret_cast<const uint2*>(a.residual + off);
      t += v4f{bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y)};
    }
    const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{t[0], t[1]}), bf2v));
    const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{t[2], t[3]}), bf2v));
    *reinterpret_cast<uint2*>(a.out + off) = make_uint2(w0, w1);
  };
  float* mine = partials + ((size_t)strip * splits + split) * a.tokens * kCols;
  for (int u = threadIdx.x; u < units; u += 64 * kMoeWaves) {
    const int t = u / (4 * FB), c = 4 * (u % (4 * FB));
    v4f v = *reinterpret_cast<const v4f*>(&sums[0][t][c]);
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) v += *reinterpret_cast<const v4f*>(&sums[w][t][c]);
    if (splits == 1) {
      finish(u, v);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) __hip_atomic_store(mine + 4 * u + q, v[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (splits == 1) return;

  // Published with device-scope atomic stores that are waited for before the barrier,
  // counted after it, and read back with device-scope atomic loads: no fence, which
  // would write back or invalidate the XCD's whole L2.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(counters + strip, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(splits - 1);
  __syncthreads();
  if (!s_last) return;
  const float* base = partials + (size_t)strip * splits * a.tokens * kCols;
  for (int u = threadIdx.x; u < units; u += 64 * kMoeWaves) {
    v4f t = v4f{0.f, 0.f, 0.f, 0.f};
    for (int sp = 0; sp < splits; ++sp) {
      const float* p = base + (size_t)sp * a.tokens * kCols + 4 * u;
#pragma unroll
      for (int q = 0; q < 4; ++q) t[q] += __hip_atomic_load(p + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    finish(u, t);
  }
  if (threadIdx.x == 0) __hip_atomic_store(counters + strip, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
constexpr int kMoeCounters = 256;

struct MoePlan {
  int fb, strips, splits;
  size_t a_bytes, bytes;
};
static MoePlan moe_plan(int tokens, int topk, int experts, int hidden, int inner) {
  MoePlan p{};
  const int nfrag = frag_rows(hidden), pairs = tokens * topk;
  p.fb = nfrag > 2 * kNumCUs ? 2 : 1;
  p.strips = nfrag / p.fb;
  p.splits = 1;
  if (p.strips <= kMoeCounters) {
    const int64_t items = (int64_t)std::min(experts, pairs) * ((inner + kBK - 1) / kBK);
    const int64_t worth = std::max<int64_t>(1, items / (2 * kMoeWaves));
    p.splits = (int)std::min<int64_t>((2 * kNumCUs + p.strips - 1) / p.strips, worth);
  }
  p.a_bytes = ((size_t)pairs * inner * 2 + 255) / 256 * 256;
  p.bytes = kMoeCounters * 4 + p.a_bytes +
            (p.splits > 1 ? (size_t)p.strips * p.splits * tokens * 16 * p.fb * sizeof(float) : 0);
  return p;
}
size_t moe_workspace_bytes(int tokens, int topk, int experts, int hidden, int inner) {
  return moe_plan(tokens, topk, experts, hidden, inner).bytes;
}

template <int XF, int WF, int MB>
static hipError_t launch_moe_up(const MoeArgs& a, int act, bool gated, hipStream_t st) {
  const int strips = gated ? a.inner / 16 : (a.inner + 31) / 32;
  const dim3 grid(std::min(a.experts, a.tokens * a.topk) * strips), block(64 * kMoeWaves);
  if (gated) hipLaunchKernelGGL((moe_up_kernel<XF, WF, MB, true>), grid, block, 0, st, a, strips, act);
  else hipLaunchKernelGGL((moe_up_kernel<XF, WF, MB, false>), grid, block, 0, st, a, strips, act);
  return hipGetLastError();
}

template <int WF, int MB, int TB>
static hipError_t launch_moe_down(const MoeArgs& a, const MoePlan& p, uint32_t* counters, float* partials, hipStream_t st) {
  const dim3 grid(p.strips * p.splits), block(64 * kMoeWaves);
  if (p.fb == 1) hipLaunchKernelGGL((moe_down_kernel<WF, MB, 1, TB>), grid, block, 0, st, a, p.splits, counters, partials);
  else hipLaunchKernelGGL((moe_down_kernel<WF, MB, 2, TB>), grid, block, 0, st, a, p.splits, counters, partials);
  return hipGetLastError();
}

template <int XF, int WF>
static hipError_t launch_moe_t(const MoeArgs& a, int act, bool gated, const MoePlan& p, uint32_t* counters, float* partials,
                               hipStream_t st) {
  // 16 rows of an expert at a time, or 32 where experts have more than 8 on average
  const bool wide = a.tokens > 16 && a.tokens * a.topk > 8 * a.experts;
  const hipError_t e = wide ? launch_moe_up<XF, WF, 2>(a, act, gated, st) : launch_moe_up<XF, WF, 1>(a, act, gated, st);
  if (e != hipSuccess) return e;
  if (a.tokens <= 16) return launch_moe_down<WF, 1, 16>(a, p, counters, partials, st);
  if (!wide) return launch_moe_down<WF, 1, 64>(a, p, counters, partials, st);
  return launch_moe_down<WF, 2, 64>(a, p, counters, partials, st);
}

hipError_t launch_moe(MoeArgs a, int xf, int wf, int act, bool gated, void* workspace, hipStream_t st) {
  const MoePlan p = moe_plan(a.tokens, a.topk, a.experts, a.hidden, a.inner);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* counters = reinterpret_cast<uint32_t*>(ws);
  a.a = reinterpret_cast<uint16_t*>(ws + kMoeCounters * 4);
  float* partials = reinterpret_cast<float*>(ws + kMoeCounters * 4 + p.a_bytes);
#define CALL(X, W) return launch_moe_t<X, W>(a, act, gated, p, counters, partials, st)
  HQ_DISPATCH_FMT_PAIR(xf, wf, CALL);
#undef CALL
}

}  // namespace hq
