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
// the logits. Up to some thousand tokens a call takes what a launch and the rounds'
// dependent lane moves take (1 token, 128 experts, topk 8: 3.6 us in a graph, bf16 3.0);
// beyond, the rounds' vector instructions bound it, not the 9.4 MB: 16384 tokens, 128
// experts, topk 8, float32 6.2 us, bf16, whose keys hold the index, 5.2 (7.0 both with
// floats compared). So are 512 and 1024 experts, and 16 slots: a wavefront has one token and
// issues some 270 vector instructions for 8 logits a lane (480 for 16) before the rounds, 52
// (88; bf16 51) and four (bf16 two) exchanges through LDS in each, and 200 after them. 16
// tokens a SIMD at 4 cycles an instruction make 16384 tokens 34 us with 512 experts, topk 16
// (29.6 measured), and 36 (bf16 29) with 1024, topk 8 (36.9 and 25.7). The backward pass
// issues some 800 with 1024 experts: 21 us (17.8).
constexpr int kMaxTopk = 16;

template <int G, class F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // swap neighbours
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // swap pairs
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // half-row mirror
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // row mirror
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
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

// A logit; NaN counts as -Inf.
template <int XT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  const float v = XT == kF32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  return v == v ? v : -__builtin_inff();
}
// A logit in the race: an unsigned integer in the logits' order (negative values' bits
// inverted, the others' sign bit set; -0 as 0), 0 for -Inf. A 16-bit logit leaves room for
// the expert below its bits, the lowest as the largest.
template <int XT>
__device__ __forceinline__ uint32_t race_key(float v, int e) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t k = b >> 31 ? ~b : b | 0x80000000u;
  return v == -__builtin_inff() ? 0u : XT == kF32 ? k : (k & 0xffff0000u) | (0xffffu - e);
}
template <int XT>
__device__ __forceinline__ float race_logit(uint32_t k) {
  if (k == 0) return -__builtin_inff();
  const uint32_t b = k >> 31 ? k & 0x7fffffffu : ~k;
  return __uint_as_float(XT == kF32 ? b : b & 0xffff0000u);
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
    uint32_t key[V], m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      key[j] = race_key<XT>(v[j], l + G * j);
      m = max(m, key[j]);
    }
    m = group_max<G>(m);
    const float top = race_logit<XT>(m);
    float all = 0.0f;  // sum of the exponentials of all experts
    if (a.score == kRouteSoftmax && !a.renormalize) {
#pragma unroll
      for (int j = 0; j < V; ++j) all += v[j] == -__builtin_inff() ? 0.0f : exp_below(v[j], top);
      all = group_sum<G>(all);
    }
    // slot r stays with lane r
    int id = -1;
    uint32_t won = 0;
    for (int r = 0; r < a.topk; ++r) {
      uint32_t at = 0xffffu - (m & 0xffffu);
      if constexpr (XT == kF32) {
        at = 0x7fffffff;
#pragma unroll
        for (int j = V - 1; j >= 0; --j) at = key[j] == m ? l + G * j : at;
        at = group_min<G>(at);
      }
      if (l == r && m != 0) {
        id = at;
        won = m;
      }
      const uint32_t best = m;
      m = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (XT == kF32 ? at == (uint32_t)(l + G * j) : key[j] == best) key[j] = 0;
        m = max(m, key[j]);
      }
      m = group_max<G>(m);
    }
    const float mine = race_logit<XT>(won);
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
// Lanes per token, measured with topk 8, float32 (us, 16 / 64 lanes): with enough tokens
// for every SIMD the instructions per token count, 16384 tokens 6.2 / 11.2 (128 experts),
// 9.2 / 12.9 (256), 17.4 / 19.4 (512), 60.7 / 36.9 (1024); with fewer the length of a
// round, 1 token 3.8 / 3.6 (128), 5.4 / 4.0 (256), 9.3 / 5.0 (512), and 64 of 64 experts
// 3.1 / 3.8, where a lane has one logit.
#define HQ_ROUTE_X(KERNEL, XT)                                  \
  do {                                                          \
    const bool few = a.tokens <= 4 * kNumCUs;                   \
    if (a.experts <= 64) HQ_ROUTE(KERNEL, XT, 16, 4);           \
    if (a.experts <= 128 && few) HQ_ROUTE(KERNEL, XT, 64, 2);   \
    if (a.experts <= 128) HQ_ROUTE(KERNEL, XT, 16, 8);          \
    if (a.experts <= 256 && few) HQ_ROUTE(KERNEL, XT, 64, 4);   \
    if (a.experts <= 256) HQ_ROUTE(KERNEL, XT, 16, 16);         \
    if (a.experts <= 512) HQ_ROUTE(KERNEL, XT, 64, 8);          \
    HQ_ROUTE(KERNEL, XT, 64, 16);                               \
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
  float x_scale[kMoeMaxTokens];
  uint32_t bits[kMoeMaxExperts / 32];
};

// Fills s, for the first kernel without the weights, for the second without the tokens'
// scales; ends with a barrier. A thread's loads are under way before the first barrier.
template <int THREADS, bool FIRST>
__device__ __forceinline__ void moe_load_pairs(const MoeArgs& a, MoeLds& s) {
  const int pairs = a.tokens * a.topk, t = threadIdx.x;
  int e = t < pairs ? a.ids[t] : -1;
  float w = !FIRST && t < pairs ? a.weights[t] : 0.0f;
  const float xs = FIRST && t < a.tokens ? a.x_scale[a.x_scale_per_row ? t : 0] : 0.0f;
  if (t < kMoeMaxExperts / 32) s.bits[t] = 0;
  __syncthreads();
  if (FIRST && t < a.tokens) s.x_scale[t] = xs;
  for (int p = t; p < pairs;) {
    s.ids[p] = e;
    if (!FIRST) s.weights[p] = w;
    if ((unsigned)e < (unsigned)a.experts) atomicOr(&s.bits[e >> 5], 1u << (e & 31));
    p += THREADS;
    if (p < pairs) {
      e = a.ids[p];
      if (!FIRST) w = a.weights[p];
    }
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
    const int own = __popc(word);
    int upto = own;  // sums of the lanes up to this one: within a row of 16 lanes, then row 0's onto row 1
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x111, 0xF, 0xF, false);
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x112, 0xF, 0xF, false);
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x114, 0xF, 0xF, false);
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x118, 0xF, 0xF, false);
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x142, 0xA, 0xF, false);
    before = upto - own;
    count = __builtin_amdgcn_readlane(upto, 31);
  }
  // The i-th of them, i < count.
  __device__ int at(int i) const {
    const uint64_t m = __ballot(before <= i && i < before + (int)__popc(word));
    const int src = __builtin_ctzll(m);
    uint32_t w = __builtin_amdgcn_readlane(word, src);
    for (int k = i - __builtin_amdgcn_readlane(before, src); k > 0; --k) w &= w - 1;
    return src * 32 + __builtin_ctz(w);
  }
};

// Activations between the kernels: bf16, the rows of an expert together, experts in
// order, K blocks of 128 padded with zeros. An expert's rows come in blocks of 16 (n in
// the last), a block's K blocks one after another, and in these the order in which the
// second kernel's lanes read: its lane of row r that has K values 32 g .. 32 g + 31 loads
// 16 bytes at a time, the m-th at ((4 m + g) n + r) 16, so that one load of a wavefront
// reads 64 n contiguous bytes (64 tokens, 64 experts of 4096 x 1408: second kernel 82.7 us;
// 92.4 with each pair's row by itself in that order, 99.6 with its columns in their own).
__host__ __device__ inline int moe_pitch(int inner) { return (inner + kBK - 1) / kBK * kBK; }
// Element of column col in row r of a block of n rows, from the block's start.
__device__ __forceinline__ int moe_place(int n, int r, int col) {
  return ((col >> 7) * 16 + (col >> 3 & 3) * 4 + (col >> 5 & 3)) * n * 8 + r * 8 + (col & 7);
}

// The tokens that chose expert e, in order, and, where wts is not null, the sum of their
// weights for it (a token that names an expert twice has one row). rows and wts have 64
// entries of this wavefront's own; before: the pairs that chose an expert below e, where the
// expert's rows of activations start.
__device__ __forceinline__ int moe_expert_rows(const MoeArgs& a, const MoeLds& s, int e, int* rows, float* wts, int& before) {
  const int t = threadIdx.x & 63;
  bool mine = false;
  int below = 0;
  float w = 0.0f;
  for (int j0 = 0; j0 < a.topk; j0 += 4) {
#pragma unroll
    for (int j = j0; j < j0 + 4; ++j) {
      const int q = t * a.topk + j;
      const int id = t < a.tokens && j < a.topk ? s.ids[q] : -1;
      below += __popcll(__ballot((unsigned)id < (unsigned)e));
      if (id == e) {
        mine = true;
        if (wts) w += s.weights[q];
      }
    }
  }
  before = below;
  const uint64_t m = __ballot(mine);
  if (mine) {
    const int at = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
    rows[at] = t;
    if (wts) wts[at] = w;
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
// A unit is two weight fragments of one expert: 16 columns of the first half and the
// same columns of the second (gated), or 32 columns. The units that the step asks for
// are dealt over the workgroups, which fill the device once, in chunks of neighbours
// (an expert with many rows takes longer: its units go to many workgroups), four chunks
// a workgroup of what is asked for: chunks of what 64 tokens could ask for left a padded
// batch of one to 102 workgroups (8 of 256 experts 2048 x 2048, call 54 us, so 30). A
// workgroup's W wavefronts take a unit's K blocks w, w + W, ... and meet in LDS at its
// end. The next block's weights and codes, also those of the next unit's first block,
// are on their way while one is multiplied. Loads return in order, so the codes travel
// with the weights: fetched when needed, they would wait for all weights in flight. Only
// an expert's rows past 16, of more than 32 tokens, are fetched that way: a second block of
// rows under way took 32 tokens, 32 experts of 7168 x 768 from 51 to 47 us, but spills with
// four (64 tokens, 64 experts of 4096 x 1408 118 -> 122). Codes are multiplied as f16, which
// holds each of them, so every product is exact and the sums are float32.
// Bound by the weights of the experts that are asked for, each read once and past the
// caches' own order (non-temporal: 117 us, else 130). 64 tokens, 64 experts of 4096 x 1408,
// 58 asked for, 669 MB: 115 us, 5.8 TB/s; 1 token, 8 of them, 92 MB: 17.7 us, 5.2 TB/s. Below
// some 10 MB a launch, the pairs and one trip to memory: 5 to 6 us.
template <int XF, int WF, int MB, bool GATED, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(MB > 1 ? 3 : 4))) void moe_up_kernel(MoeArgs a, int strips, int act) {
  // two buffers for the sums save a barrier; with more row blocks they would cost a workgroup per CU
  constexpr int kBufs = W > 1 && MB == 1 ? 2 : 1;
  __shared__ MoeLds s;
  __shared__ int s_rows[2][W][kMoeMaxTokens];  // of two experts in turn
  __shared__ __attribute__((aligned(16))) v4f red[kBufs][W > 1 ? W : 1][W > 1 ? 2 * MB : 1][64];
  constexpr int PB = MB == 2 ? 2 : 1;  // blocks of rows whose codes travel with the weights
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  moe_load_pairs<64 * W, true>(a, s);
  const ActiveExperts active(s);
  const int all = active.count * strips;
  const int chunk = max(1, all / (4 * (int)gridDim.x));
  if ((int)blockIdx.x * chunk >= all) return;

  const int K = a.hidden, nkb = (K + kBK - 1) / kBK;
  const int n1 = GATED ? 2 * a.inner : a.inner;
  const size_t w_bytes = (size_t)frag_rows(n1) * nkb * kFragBytes;
  const __amdgpu_buffer_rsrc_t x_rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)a.xq, (short)0, a.tokens * K, kRsrcFlags);
  const int xr = lane & 15, xc = 32 * (lane >> 4);
  auto fragment = [&](int f, int strip) { return GATED ? (f ? a.inner / 16 + strip : strip) : 2 * strip + f; };

  struct Unit {
    int at, slot, strip, e, rows, list, before;
  };
  __amdgpu_buffer_rsrc_t w_rsrc[2];
  auto row_offset = [&](const Unit& u, int i) {
    const int r = 16 * i + xr;
    return r < u.rows ? s_rows[u.list][wave][r] * K + xc : kBadOffset;
  };
  int xo[PB];  // the lane's rows of the first blocks
  auto enter = [&](Unit& u) {
    const int slot = u.at / strips;
    u.strip = u.at - slot * strips;
    if (slot != u.slot) {
      u.slot = slot;
      u.e = active.at(slot);
      u.list ^= 1;
      u.rows = moe_expert_rows(a, s, u.e, s_rows[u.list][wave], nullptr, u.before);
#pragma unroll
      for (int i = 0; i < PB; ++i) xo[i] = row_offset(u, i);
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
      w_rsrc[f] = __builtin_amdgcn_make_buffer_rsrc((void*)(a.w1 + u.e * w_bytes + (size_t)fragment(f, u.strip) * nkb * kFragBytes),
                                                    (short)0, nkb * kFragBytes, kRsrcFlags);
  };
  auto load_x = [&](uint4 (&x)[2], int off, int kb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = kb * kBK + 16 * h;
      x[h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(x_rsrc, col + xc < K && off >= 0 ? off + col : kBadOffset, 0, 0));
    }
  };
  struct Chunk {
    uint4 w[2][2], x[PB][2];
  };
  auto load = [&](Chunk& c, int kb) {
    const int wo = kb < nkb ? lane * 16 : kBadOffset;  // the scalar offset is not range-checked
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        c.w[f][h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(w_rsrc[f], wo + h * 1024, min(kb, nkb - 1) * kFragBytes, kNtLoad));
#pragma unroll
    for (int i = 0; i < PB; ++i) load_x(c.x[i], xo[i], kb);
    __builtin_amdgcn_sched_barrier(0);  // ahead of the products that follow
  };

  v4f acc[2][MB];
  Unit cur;
  auto multiply = [&](const Chunk& c, int kb) {
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      uint4 late[2];
      if (i > 0 && 16 * i >= cur.rows) break;  // wavefront-uniform
      if (i >= PB) load_x(late, row_offset(cur, i), kb);
      const uint4(&x)[2] = i >= PB ? late : c.x[i < PB ? i : 0];
      // 8 values of K per lane at a time: few converted codes are alive
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4& xs = x[q >> 1];
        const h8v xh = q & 1 ? f16x8<XF>(xs.z, xs.w) : f16x8<XF>(xs.x, xs.y);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint4& ws = c.w[f][q >> 1];
          const h8v wh = q & 1 ? f16x8<WF>(ws.z, ws.w) : f16x8<WF>(ws.x, ws.y);
          acc[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh, xh, acc[f][i], 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  constexpr int kParts = GATED ? MB : 2 * MB;  // 16 rows (gated), or one fragment of them
  int parity = 0, turn = 0;
  float sc[2][4];
  // Scales of the lane's 4 columns of each fragment.
  auto load_scales = [&]() {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int nb = fragment(f, cur.strip);
      const int col = 32 * (nb >> 1) + 8 * (lane >> 4) + 4 * (nb & 1);
#pragma unroll
      for (int q = 0; q < 4; ++q) sc[f][q] = a.s1[a.s1_per_col ? (size_t)cur.e * n1 + min(col + q, n1 - 1) : cur.e];
    }
  };
  auto finish = [&]() {
    if constexpr (W > 1) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int i = 0; i < MB; ++i)
          if (16 * i < cur.rows) red[parity][wave][f * MB + i][lane] = acc[f][i];
      __syncthreads();
    }
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      const int i = GATED ? part : part >> 1;
      if ((W > 1 && (part + turn) % W != wave) || 16 * i >= cur.rows) continue;
      const int r = 16 * i + xr;
      const float xs = s.x_scale[s_rows[cur.list][wave][min(r, cur.rows - 1)]];
      float z[2][4];
#pragma unroll
      for (int f = 0; f < (GATED ? 2 : 1); ++f) {
        const int ff = GATED ? f : part & 1;
        v4f t;
        if constexpr (W == 1) {
          t = acc[ff][i];
        } else {
          t = red[parity][0][ff * MB + i][lane];
#pragma unroll
          for (int v = 1; v < W; ++v) t += red[parity][v][ff * MB + i][lane];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) z[f][q] = t[q] * xs * sc[ff][q];
        if (a.b1) {
          const int nb = fragment(ff, cur.strip);
          const int col = 32 * (nb >> 1) + 8 * (lane >> 4) + 4 * (nb & 1);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            z[f][q] += __uint_as_float((uint32_t)a.b1[(size_t)cur.e * n1 + min(col + q, n1 - 1)] << 16);
        }
      }
      float o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = z[0][q];
      fused_act<4>(act, o);
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] *= z[1][q];
      }
      const int nb = fragment(GATED ? 0 : part & 1, cur.strip);
      const int col = 32 * (nb >> 1) + 8 * (lane >> 4) + 4 * (nb & 1);
      if (r < cur.rows) {
        const int n = min(16, cur.rows - 16 * i);
        uint16_t* block = a.a + (size_t)(cur.before + 16 * i) * moe_pitch(a.inner);
        const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{o[0], o[1]}), bf2v));
        const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{o[2], o[3]}), bf2v));
        if (col < a.inner) *reinterpret_cast<uint2*>(block + moe_place(n, xr, col)) = make_uint2(w0, w1);
        if (cur.strip + 1 == strips)  // the row's end is zeros
          for (int z = a.inner + 4 * (lane >> 4); z < moe_pitch(a.inner); z += 16)
            *reinterpret_cast<uint2*>(block + moe_place(n, xr, z)) = make_uint2(0u, 0u);
      }
    }
    if constexpr (kBufs == 2) parity ^= 1;
    else if constexpr (W > 1) __syncthreads();
    turn = (turn + kParts) % W;
  };

  Unit next{(int)blockIdx.x * chunk, -1, 0, 0, 0, 0, 0};
  enter(next);
  Chunk c0, c1;
  load(c0, wave);
  int in_chunk = 0;
  for (;;) {
    cur = next;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < MB; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb = wave;; kb += 2 * W) {
      const bool more = kb + W < nkb;
      if (more) load(c1, kb + W);
      if (MB == 1 && kb == wave) load_scales();  // (more row blocks have no registers for them)
      multiply(c0, kb);
      if (!more) break;
      const bool again = kb + 2 * W < nkb;
      if (again) load(c0, kb + 2 * W);
      multiply(c1, kb + W);
      if (!again) break;
    }
    if (MB > 1) load_scales();
    if (++in_chunk == chunk) {
      in_chunk = 0;
      next.at += (int)(gridDim.x - 1) * chunk;
    }
    const bool more = ++next.at < all;
    if (more) {
      enter(next);
      load(c0, wave);
    }
    finish();
    if (!more) return;
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

// A workgroup owns one weight fragment (16 output columns) of every expert, and all
// tokens; the (expert, K block) items are dealt in runs over its W wavefronts and over
// `splits` workgroups. The next item's operands are on their way while one is
// multiplied; an expert's rows past 16 are all fetched when they are (at 17 to 32 tokens
// 120 of 128 registers are taken, a second block under way has 16; past 32 tokens 12 bytes a
// lane are in scratch memory as it is). A wavefront adds an expert's weighted rows into
// sums of its own in LDS ([token][column], 16 MB tokens), so no two lanes meet; at the end
// the wavefronts' sums are added in order, and with splits > 1 the last workgroup to
// arrive adds the workgroups' sums, in order too: the result does not depend on who ends
// first.
// The activations are bf16, as is this product: float32's range (a gated activation passes
// what f16 holds) in half the bytes, at half a step, 2^-8, of each term. Error against 64
// bits, relative to the result's norm: 0.0023 with it, 0.0017 (the output's own rounding)
// with float32 activations. Sums are float32.
// Bound by the weights up to 16 tokens (56 of the 64 experts above, 323 MB: 53 us, 6.1 TB/s;
// 1 token, 46 MB: 10.6 us). With more rows per expert the activations, which every
// workgroup reads from L2, reach the weights' bytes: 64 tokens, 335 MB of weights and 380 of
// activations, 82 us. Two fragments per item halve them, 75 us there, but leave 8
// wavefronts per CU: 7168 x 768 35 -> 50 us, 256 x 2048 19 -> 29.
template <int WF, int MB, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(4))) void moe_down_kernel(MoeArgs a, int splits,
                                                                                                     uint32_t* counters, float* partials) {
  constexpr int TB = 16 * MB, kPitch = 20;
  __shared__ MoeLds s;
  __shared__ int s_rows[2][W][kMoeMaxTokens];
  __shared__ float s_wts[2][W][kMoeMaxTokens];
  __shared__ __attribute__((aligned(16))) float sums[W][TB][kPitch];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strip = blockIdx.x / splits, split = blockIdx.x % splits;
  moe_load_pairs<64 * W, false>(a, s);
  const ActiveExperts active(s);

  const int K = a.inner, nkb = (K + kBK - 1) / kBK;
  const int nfrag = frag_rows(a.hidden);
  const int xr = lane & 15, xq = lane >> 4;
  const int col0 = 32 * (strip >> 1) + 8 * xq + 4 * (strip & 1);  // the lane's 4 columns
  // At the end a thread has 4 columns of a token; what is added to them is fetched now.
  const int t_end = threadIdx.x >> 2, col_end = 32 * (strip >> 1) + 8 * (threadIdx.x & 3) + 4 * (strip & 1);
  const bool ends = t_end < a.tokens && col_end < a.hidden;
  uint2 res = make_uint2(0u, 0u);
  if (a.residual && ends) res = *reinterpret_cast<const uint2*>(a.residual + (size_t)t_end * a.hidden + col_end);
  const __amdgpu_buffer_rsrc_t a_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)a.a, (short)0, a.tokens * a.topk * moe_pitch(K) * 2, kRsrcFlags);
  const int64_t items = (int64_t)active.count * nkb;
  const int runs = splits * W, run = split * W + wave;
  const int first = (int)(items * run / runs), last = (int)(items * (run + 1) / runs);

  auto clear_sums = [&]() {  // the wavefront's own
    for (int i = lane; i < a.tokens * (kPitch / 4); i += 64)
      *reinterpret_cast<v4f*>(&sums[wave][0][0] + 4 * i) = v4f{0.f, 0.f, 0.f, 0.f};
  };
  if (first >= last) {
    clear_sums();
  } else {
    struct Segment {  // a run's items of one expert: K blocks kb0 .. kb1 - 1
      int slot, e, rows, list, before, kb0, kb1;
    };
    __amdgpu_buffer_rsrc_t w_rsrc;
    struct Rows {  // a block of rows: the lane's place in a K block, the first of these, their size
      int lane_at, at, size;
    };
    auto block_rows = [&](const Segment& g, int i) {
      const int n = min(16, g.rows - 16 * i);
      return Rows{xr < n ? (xq * n + xr) * 16 : kBadOffset, (g.before + 16 * i) * moe_pitch(K) * 2, n * 2 * kBK};
    };
    Rows ao;
    auto enter = [&](Segment& g, int at) {
      g.kb1 = min(nkb, g.kb0 + last - at);
      g.e = active.at(g.slot);
      g.list ^= 1;
      g.rows = moe_expert_rows(a, s, g.e, s_rows[g.list][wave], s_wts[g.list][wave], g.before);
      ao = block_rows(g, 0);
      w_rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)(a.w2 + ((size_t)g.e * nfrag + strip) * nkb * kFragBytes), (short)0,
                                                 nkb * kFragBytes, kRsrcFlags);
    };
    auto load_a = [&](uint4 (&v)[4], const Rows& b, int kb) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
        v[m] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(a_rsrc, b.lane_at, b.at + kb * b.size + m * (b.size >> 2), 0));
    };
    struct Chunk {
      uint4 w[2], v[4];
    };
    auto load = [&](Chunk& c, int kb) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        c.w[h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(w_rsrc, lane * 16 + h * 1024, kb * kFragBytes, 0));
      load_a(c.v, ao, kb);
      __builtin_amdgcn_sched_barrier(0);  // ahead of the products that follow
    };
    v4f acc[MB];
    float sc[4];
    Segment cur;
    auto multiply = [&](const Chunk& c, int kb) {
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        uint4 late[4];
        if (i > 0) {
          if (16 * i >= cur.rows) break;  // wavefront-uniform
          load_a(late, block_rows(cur, i), kb);
        }
        const uint4(&v)[4] = i > 0 ? late : c.v;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint4& ws = c.w[m >> 1];
          const b8v w = m & 1 ? bf16x8<WF>(ws.z, ws.w) : bf16x8<WF>(ws.x, ws.y);
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(b8v, v[m]), acc[i], 0, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto load_scales = [&]() {
#pragma unroll
      for (int q = 0; q < 4; ++q) sc[q] = a.s2[a.s2_per_col ? (size_t)cur.e * a.hidden + min(col0 + q, a.hidden - 1) : cur.e];
    };
    Segment next{first / nkb, 0, 0, 0, 0, 0, 0};
    next.kb0 = first - next.slot * nkb;
    int at = first;  // first item of the segment
    enter(next, at);
    Chunk c0, c1;
    load(c0, next.kb0);
    clear_sums();
    for (;;) {
      cur = next;
#pragma unroll
      for (int i = 0; i < MB; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
      for (int kb = cur.kb0;; kb += 2) {
        const bool more = kb + 1 < cur.kb1;
        if (more) load(c1, kb + 1);
        if (MB == 1 && kb == cur.kb0) load_scales();  // (more row blocks have no registers for them)
        multiply(c0, kb);
        if (!more) break;
        const bool again = kb + 2 < cur.kb1;
        if (again) load(c0, kb + 2);
        multiply(c1, kb + 1);
        if (!again) break;
      }
      if (MB > 1) load_scales();
      at += cur.kb1 - cur.kb0;
      const bool more = at < last;
      if (more) {
        ++next.slot;
        next.kb0 = 0;
        enter(next, at);
        load(c0, 0);
      }
      // lane l holds row l % 16 and 4 columns
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int r = 16 * i + xr;
        if (r >= cur.rows) continue;
        const float wt = s_wts[cur.list][wave][r];
        v4f* p = reinterpret_cast<v4f*>(&sums[wave][s_rows[cur.list][wave][r]][4 * xq]);
        v4f t = *p;
        const bool biased = a.b2 && cur.kb0 == 0;  // with the expert's first K block
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y = acc[i][q] * sc[q];
          if (biased) y += __uint_as_float((uint32_t)a.b2[(size_t)cur.e * a.hidden + min(col0 + q, a.hidden - 1)] << 16);
          t[q] = fmaf(wt, y, t[q]);
        }
        *p = t;
      }
      if (!more) break;
    }
  }
  __syncthreads();

  auto finish = [&](v4f t) {
    t += v4f{bf16_lo(res.x), bf16_hi(res.x), bf16_lo(res.y), bf16_hi(res.y)};
    const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{t[0], t[1]}), bf2v));
    const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{t[2], t[3]}), bf2v));
    *reinterpret_cast<uint2*>(a.out + (size_t)t_end * a.hidden + col_end) = make_uint2(w0, w1);
  };
  const size_t part = (size_t)a.tokens * 16;  // floats of a workgroup's sums
  float* base = partials + (size_t)strip * splits * part + 4 * threadIdx.x;
  if (ends) {
    const float* p = &sums[0][t_end][4 * (threadIdx.x & 3)];
    v4f v = *reinterpret_cast<const v4f*>(p);
#pragma unroll
    for (int w = 1; w < W; ++w) v += *reinterpret_cast<const v4f*>(p + w * TB * kPitch);
    if (splits == 1) {
      finish(v);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) __hip_atomic_store(base + split * part + q, v[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
  if (ends) {
    v4f t = v4f{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < splits; s0 += 8) {  // 8 loads in flight; added in order
      v4f v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* p = base + min(s0 + i, splits - 1) * part;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[i][q] = __hip_atomic_load(p + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s0 + i < splits) t += v[i];
    }
    finish(t);
  }
  if (threadIdx.x == 0) __hip_atomic_store(counters + strip, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
constexpr int kMoeCounters = 256;

// The second kernel's workgroups: `strips` fragments times `splits`, of `waves`
// wavefronts; 16 wavefronts per CU where the items suffice for four each. One workgroup of
// 16 wavefronts fits on a CU, so there are never more of them than CUs: the few past the
// device would take as long again (32 experts of hidden x 1536, top 4, call in a graph, us,
// at most / at least 256 workgroups: 16 tokens 768 24.8 / 28.9, 1040 28.0 / 35.5, 2080
// 39.5 / 47.7, 3584 63.7 / 69.3; 64 tokens 44.9 / 51.3, 48.3 / 60.3, 79.1 / 100.6, 85.4 / 103.7;
// 1024, 2048 and 4096 are the same in both). (Second kernel,
// us, for two / four / sixteen each: 13 tokens, 24 of 1040 x 368 9.0 / 8.1 / 8.1; 2 tokens, 8 of
// 2048 x 2048 7.6 / 6.7 / 6.7; 16 tokens, 128 of 512 x 512 10.0 / 10.0 / 13.2; 64 tokens, 8 of
// 2048 x 2048 17.3 / 17.2 / 20.0.)
struct MoePlan {
  int strips, splits, waves;
  size_t a_bytes, bytes;
};
static MoePlan moe_plan(int tokens, int topk, int experts, int hidden, int inner) {
  MoePlan p{};
  const int pairs = tokens * topk;
  p.strips = frag_rows(hidden);
  p.waves = p.strips > kNumCUs ? 8 : 16;
  p.splits = 1;
  if (p.strips < kNumCUs) {
    const int64_t items = (int64_t)std::min(experts, pairs) * ((inner + kBK - 1) / kBK);
    const int64_t worth = std::max<int64_t>(1, items / (4 * p.waves));
    p.splits = (int)std::min<int64_t>(kNumCUs / p.strips, worth);
  }
  p.a_bytes = (size_t)pairs * moe_pitch(inner) * 2;
  p.bytes = kMoeCounters * 4 + p.a_bytes + (p.splits > 1 ? (size_t)p.strips * p.splits * tokens * 16 * sizeof(float) : 0);
  return p;
}
size_t moe_workspace_bytes(int tokens, int topk, int experts, int hidden, int inner) {
  return moe_plan(tokens, topk, experts, hidden, inner).bytes;
}

template <int XF, int WF, int MB, int W>
static hipError_t launch_moe_up_w(const MoeArgs& a, int act, bool gated, int strips, int units, hipStream_t st) {
  // As many as the registers hold at once: 16 or 12 wavefronts per CU. (Past 32 tokens workgroups
  // of 8 wavefronts fit once on a CU, and up to 128 of them take the places of those that end. With
  // 256, us for 64 tokens of 8 experts: 7168 x 768 41.4 -> 51.6, 4096 x 640 28.3 -> 30.5, 2048 x 992
  // 24.4 -> 23.1.)
  constexpr int kResident = (MB > 1 ? 12 : 16) * kNumCUs / W;
  const int groups = std::min(units, kResident);
  if (gated) hipLaunchKernelGGL((moe_up_kernel<XF, WF, MB, true, W>), dim3(groups), dim3(64 * W), 0, st, a, strips, act);
  else hipLaunchKernelGGL((moe_up_kernel<XF, WF, MB, false, W>), dim3(groups), dim3(64 * W), 0, st, a, strips, act);
  return hipGetLastError();
}

// Wavefronts per unit: enough K blocks for two or more each, and enough wavefronts for the
// device where units are few. Measured (call in a graph, us, with 1 / 2 / 4 / 8): 16 of 128
// experts 512 x 512 18.1 / 18.3 / 20.5 / 26.9; 40 tokens, 100 experts 256 x 2048 34.9 / 38.3 /
// 49.1 / 113; 64 tokens, 8 experts 2048 x 2048 46.3 / 41.3 / 36.5 / 44.5; 64 experts 4096 x 1408,
// 1 token (704 units) 33.0 / 29.1 / 29.0 / 28.8 and 64 tokens 220 / 204 / 194 / 237; 1 token, 32
// experts 7168 x 768 (192 units) 36.7 / 25.6 / 20.2 / 18.2. At 17 to 32 tokens a CU holds one
// workgroup of 8 or three of 4, which are ahead where the units are more than the CUs (4 / 8,
// 32 tokens of 8 experts: 320 units 4096 x 640 19.8 / 22.7; 384 units 2048 x 768 14.9 / 18.0, 7168 x
// 768 31.9 / 34.0; 192 units 7168 x 384 20.9 / 19.7). Past 32 tokens neither is ahead between one
// and two units per CU (2048 x 992 22.4 / 24.4, 3584 x 768 29.6 / 27.2, 7168 x 768 55.0 / 41.4).
template <int XF, int WF, int MB>
static hipError_t launch_moe_up(const MoeArgs& a, int act, bool gated, hipStream_t st) {
  const int strips = gated ? a.inner / 16 : (a.inner + 31) / 32;
  const int units = std::min(a.experts, a.tokens * a.topk) * strips;
  const int nkb = (a.hidden + kBK - 1) / kBK;
  if (nkb <= 2) return launch_moe_up_w<XF, WF, MB, 1>(a, act, gated, strips, units, st);
  if (nkb <= 4) return launch_moe_up_w<XF, WF, MB, 2>(a, act, gated, strips, units, st);
  if (units >= (MB == 2 ? kNumCUs + 1 : 2 * kNumCUs) || nkb <= 8) return launch_moe_up_w<XF, WF, MB, 4>(a, act, gated, strips, units, st);
  return launch_moe_up_w<XF, WF, MB, 8>(a, act, gated, strips, units, st);
}

template <int WF, int MB>
static hipError_t launch_moe_down(const MoeArgs& a, const MoePlan& p, uint32_t* counters, float* partials, hipStream_t st) {
  const dim3 grid(p.strips * p.splits), block(64 * p.waves);
  if (p.waves == 8) hipLaunchKernelGGL((moe_down_kernel<WF, MB, 8>), grid, block, 0, st, a, p.splits, counters, partials);
  else hipLaunchKernelGGL((moe_down_kernel<WF, MB, 16>), grid, block, 0, st, a, p.splits, counters, partials);
  return hipGetLastError();
}

// Row blocks of 16 that a kernel holds: as many as the step has tokens.
template <int XF, int WF, int MB>
static hipError_t launch_moe_m(const MoeArgs& a, int act, bool gated, const MoePlan& p, uint32_t* counters, float* partials,
                               hipStream_t st) {
  const hipError_t e = launch_moe_up<XF, WF, MB>(a, act, gated, st);
  return e != hipSuccess ? e : launch_moe_down<WF, MB>(a, p, counters, partials, st);
}
template <int XF, int WF>
static hipError_t launch_moe_t(const MoeArgs& a, int act, bool gated, const MoePlan& p, uint32_t* counters, float* partials,
                               hipStream_t st) {
  if (a.tokens <= 16) return launch_moe_m<XF, WF, 1>(a, act, gated, p, counters, partials, st);
  if (a.tokens <= 32) return launch_moe_m<XF, WF, 2>(a, act, gated, p, counters, partials, st);
  return launch_moe_m<XF, WF, 4>(a, act, gated, p, counters, partials, st);
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
