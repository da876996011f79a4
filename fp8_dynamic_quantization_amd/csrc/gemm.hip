// Scaled FP8 (a8w8) GEMM, its grouped and block-scaled forms and the weight
// pre-shuffle, gfx950. The tile, the weight-streaming kernel and their launch
// rules are in gemm_kernels.h.
#include "gemm_kernels.h"

#include <mutex>

namespace hq {

// ---------------------------------------------------------------------------
// pre-shuffle
// ---------------------------------------------------------------------------
// One thread per 16-byte piece of the output. Piece P of fragment (nb, kb):
// h = P / 64, slot = P % 16, quarter q = (P % 64) / 16 -> weight row
// 32*(nb/2) + 8*(slot/4) + 4*(nb%2) + slot%4, columns kb*128 + 32*q + 16*h .. +15.
__global__ __launch_bounds__(256) void preshuffle_kernel(const uint8_t* __restrict__ wq, int n, int k, int kblocks,
                                                         size_t npieces, uint8_t* __restrict__ out) {
  const size_t pc = blockIdx.x * (size_t)256 + threadIdx.x;
  if (pc >= npieces) return;
  const size_t frag = pc / 128;
  const int p = (int)(pc % 128);
  const int h = p / 64, q = (p % 64) / 16, slot = p % 16;
  const int nb = (int)(frag / kblocks), kb = (int)(frag % kblocks);
  const int row = 32 * (nb >> 1) + 8 * (slot >> 2) + 4 * (nb & 1) + (slot & 3);
  const int col = kb * kBK + q * 32 + h * 16;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (row < n && col < k) v = *reinterpret_cast<const uint4*>(wq + (size_t)row * k + col);
  *reinterpret_cast<uint4*>(out + pc * 16) = v;
}

hipError_t launch_preshuffle(const uint8_t* wq, int n, int k, uint8_t* out, hipStream_t st) {
  const int kblocks = (k + kBK - 1) / kBK;
  const size_t npieces = (size_t)frag_rows(n) * kblocks * 128;
  const size_t grid = (npieces + 255) / 256;
  hipLaunchKernelGGL(preshuffle_kernel, dim3((unsigned)grid), dim3(256), 0, st, wq, n, k, kblocks, npieces, out);
  return hipGetLastError();
}

// Block-scaled form (blocks of 128 along K) on the same data path.
template <int XF, int WF, int BM, int TN, int WM, bool KTAIL, int BSZ>
__global__ __launch_bounds__(256 * WM) __attribute__((amdgpu_waves_per_eu(2))) void gemm_bsf_kernel(GemmArgs a, int tiles_m, int tiles_n) {
  using C = BsCfg<BM, TN, WM>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLdsBytes + C::kBsfBytes * (128 / BSZ)];
  int tm, tn;
  tile_coords(xcd_remap(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * BM;
  gemm_tile<XF, WF, BM, TN, WM, KTAIL, BSZ>(a, lds, m0, min(a.m, m0 + BM), tn * C::kBN, a.wq_pre, a.w_scale);
}

// Grouped: a linear tile id enumerates, per expert in order, its row tiles x the
// column tiles. Offsets are clamped so any input stays in bounds.
template <int XF, int WF, int BM, int TN, int WM, bool KTAIL, bool STRICT>
__global__ __launch_bounds__(256 * WM) void grouped_gemm_kernel(GemmArgs a, const int32_t* offsets, int experts,
                                                                int tiles_n, size_t expert_bytes) {
  using C = BsCfg<BM, TN, WM>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLdsBytes];
  __shared__ int s_sel[3];  // expert, first row, row end
  const int t = xcd_remap(blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) {
    const int tm_target = t / tiles_n;
    int acc = 0, lo = 0;
    s_sel[0] = -1;
    for (int e = 0; e < experts; ++e) {
      // clamp to [previous end, m] so the ranges are disjoint and in bounds
      const int b = min(max(offsets[e], lo), a.m);
      const int end = min(max(offsets[e + 1], b), a.m);
      lo = end;
      const int cnt = (end - b + BM - 1) / BM;
      if (tm_target < acc + cnt) {
        s_sel[0] = e;
        s_sel[1] = b + (tm_target - acc) * BM;
        s_sel[2] = end;
        break;
      }
      acc += cnt;
    }
  }
  __syncthreads();
  const int e = s_sel[0];
  if (e < 0) return;
  const int m0 = s_sel[1];
  const int row_end = min(s_sel[2], m0 + BM);
  const int tn = t % tiles_n;
  const float* ws = a.w_scale + (size_t)e * (a.w_scale_per_col ? a.n : 1);
  // the epilogue's bias is per expert: [experts, n] values, and an FP8 bias has
  // one bias scale per expert; the output scale is shared
  GemmArgs ae = a;
  if (a.bias) {
    ae.bias = static_cast<const uint8_t*>(a.bias) + (size_t)e * a.n * (a.bias_kind == kBiasBF16 ? 2 : 1);
    if (a.bias_scale) ae.bias_scale = a.bias_scale + e;
  }
  gemm_tile<XF, WF, BM, TN, WM, KTAIL, 0, STRICT>(ae, lds, m0, row_end, tn * C::kBN, a.wq_pre + e * expert_bytes, ws);
}

SkinnyPlan skinny_plan(int m, int n, int k) {
  SkinnyPlan p{};
  p.mb = m <= 16 ? 1 : (m <= 32 ? 2 : 4);
  p.f = p.mb == 1 ? 1 : 2;
  p.kpw = p.mb == 1 ? 4 : (p.mb == 2 ? 2 : 1);  // loads in flight within the 128-VGPR budget
  p.groups = (frag_rows(n) + p.f - 1) / p.f;
  p.halves = 1;
  // One 16-row activation block and fewer fragments than CUs: each fragment's
  // two slot halves go to two workgroups (the other half's lanes load zeros),
  // so every CU streams weight with no cross-workgroup sum.
  if (p.mb == 1 && p.groups < 256) {
    p.halves = 2;
    p.groups *= 2;
  }
  // Split only when one workgroup per group would take its wavefronts through
  // more than one chunk of loads: below that the cross-workgroup step costs
  // more latency than the extra workgroups save.
  p.splits = 1;
  const int nkb = (k + kBK - 1) / kBK;
  p.kb = nkb;
  if (nkb > kSkWaves * p.kpw && p.groups < (int)(kSkCounterBytes / 4)) {
    while (p.splits < 8 && p.groups * p.splits < 256) p.splits *= 2;
    while (p.splits > 1 && nkb < p.splits * 2) p.splits /= 2;  // at least 2 K blocks per workgroup
  }
  p.workspace_bytes = p.splits == 1 ? 0 : kSkCounterBytes + (size_t)p.groups * p.splits * p.f * p.mb * 1024;
  // Wavefronts per fragment group: 16 for split plans; unsplit, the next power
  // of two of ceil(nkb / 8), at least 2 (each wavefront then takes up to 8 K
  // blocks, two chunks of loads). Smaller workgroups cost less to start and
  // reduce: N = 7168, K = 768 / 2048, M = 1 (one weight copy): 7.9 / 8.2 us at
  // 16 wavefronts, 3.1 / 3.9 us at 2; N = 2048, K = 7168: 6.7 us at 16, 6.55 at 8.
  p.waves = kSkWaves;
  if (p.splits == 1) {
    int w = 2;
    while (w < kSkWaves && w * 8 < nkb) w *= 2;
    p.waves = w;
  }
  return p;
}

template <int XF, int WF, int BM, int TN, int WM, bool STRICT>
static hipError_t launch_grouped_cfg(const GemmArgs& a, const int32_t* offsets, int experts, hipStream_t st) {
  using C = BsCfg<BM, TN, WM>;
  const int tiles_n = (a.n + C::kBN - 1) / C::kBN;
  const int tiles_m = (a.m + BM - 1) / BM + experts;  // bound for any clamped offsets
  const size_t expert_bytes = (size_t)frag_rows(a.n) * 16 * (size_t)((a.k + kBK - 1) / kBK * kBK);
  if (a.k % kBK == 0)
    hipLaunchKernelGGL((grouped_gemm_kernel<XF, WF, BM, TN, WM, false, STRICT>), dim3(tiles_m * tiles_n),
                       dim3(C::kThreads), 0, st, a, offsets, experts, tiles_n, expert_bytes);
  else
    hipLaunchKernelGGL((grouped_gemm_kernel<XF, WF, BM, TN, WM, true, STRICT>), dim3(tiles_m * tiles_n),
                       dim3(C::kThreads), 0, st, a, offsets, experts, tiles_n, expert_bytes);
  return hipGetLastError();
}

// Block-scaled form: 256 x 128, 128 x 128 or 64 x 128 tiles (64 accumulators
// per wavefront, room for the fold's sums and scales), chosen by the cost rule
// of pick_tile with their measured relative throughputs (0.83, 0.81, 0.67 of the
// plain 256 x 256 tile).
template <int XF, int WF, int BM, int TN, int WM, int BSZ>
static hipError_t launch_bsf_cfg(const GemmArgs& a, hipStream_t st) {
  using C = BsCfg<BM, TN, WM>;
  const int tiles_m = (a.m + BM - 1) / BM, tiles_n = (a.n + C::kBN - 1) / C::kBN;
  if (a.k % kBK == 0)
    hipLaunchKernelGGL((gemm_bsf_kernel<XF, WF, BM, TN, WM, false, BSZ>), dim3(tiles_m * tiles_n), dim3(C::kThreads), 0,
                       st, a, tiles_m, tiles_n);
  else
    hipLaunchKernelGGL((gemm_bsf_kernel<XF, WF, BM, TN, WM, true, BSZ>), dim3(tiles_m * tiles_n), dim3(C::kThreads), 0,
                       st, a, tiles_m, tiles_n);
  return hipGetLastError();
}

template <int XF, int WF, int BSZ>
static hipError_t launch_bsf_t(const GemmArgs& a, hipStream_t st) {
  const struct {
    int bm;
    double eff;
  } cands[] = {{256, 0.83}, {128, 0.81}, {64, 0.67}};
  int best = 0;
  double best_cost = 0.0;
  for (int c = 0; c < 3; ++c) {
    const long tiles = (long)((a.m + cands[c].bm - 1) / cands[c].bm) * ((a.n + 127) / 128);
    const double cost = (double)((tiles + kNumCUs - 1) / kNumCUs) * cands[c].bm * 128 / cands[c].eff;
    if (c == 0 || cost < best_cost) {
      best = c;
      best_cost = cost;
    }
  }
  if (best == 0) return launch_bsf_cfg<XF, WF, 256, 32, 2, BSZ>(a, st);
  if (best == 1) return launch_bsf_cfg<XF, WF, 128, 32, 1, BSZ>(a, st);
  return launch_bsf_cfg<XF, WF, 64, 32, 1, BSZ>(a, st);
}

template <int XF, int WF, bool STRICT>
static hipError_t launch_grouped_s(const GemmArgs& a, const int32_t* offsets, int experts, hipStream_t st) {
  if (pick_tile(a.m, a.n, experts, STRICT) == kTile128)
    return launch_grouped_cfg<XF, WF, 128, 32, 1, STRICT>(a, offsets, experts, st);
  return launch_grouped_cfg<XF, WF, 64, 32, 1, STRICT>(a, offsets, experts, st);
}

template <int XF, int WF>
static hipError_t launch_grouped_t(const GemmArgs& a, const int32_t* offsets, int experts, hipStream_t st) {
  return a.strict ? launch_grouped_s<XF, WF, true>(a, offsets, experts, st)
                  : launch_grouped_s<XF, WF, false>(a, offsets, experts, st);
}

// ---------------------------------------------------------------------------
// library-held scratch (hq_gemm_a8w8_noalloc)
// ---------------------------------------------------------------------------
// For callers that cannot allocate device memory (code under HIP graph
// capture, tight serving loops), split decode launches take their workspace
// from this file-scope device array instead of a caller buffer. Each GPU holds
// its own copy until the process ends; host code reaches it only through the
// per-device address from hipGetSymbolAddress (the array's name in host code is
// a host-side stand-in, not a device address). The counter region is zeroed
// once per device at set-up, by a small kernel on the caller's stream, and every
// launch leaves it at zero; the partial sums need no reset. Every call on a GPU
// shares that GPU's array, so calls that overlap on one GPU race on it.
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];

__global__ __launch_bounds__(256) void zero_words_kernel(uint32_t* p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0u;
}

hipError_t noalloc_scratch(hipStream_t st, void** ptr) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  static std::mutex mu;
  static void* addr[kMaxDevices];
  std::lock_guard<std::mutex> lk(mu);
  if (addr[dev] == nullptr) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    constexpr int words = (int)(kSkCounterBytes / 4);
    hipLaunchKernelGGL(zero_words_kernel, dim3((words + 255) / 256), dim3(256), 0, st, static_cast<uint32_t*>(p), words);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    addr[dev] = p;
  }
  *ptr = addr[dev];
  return hipSuccess;
}

size_t gemm_workspace_bytes(int m, int n, int k) {
  return m >= 1 && m <= kSkinnyMaxM ? skinny_plan(m, n, k).workspace_bytes : 0;
}

hipError_t launch_gemm(const GemmArgs& a, int xf, int wf, void* workspace, size_t workspace_bytes, hipStream_t st) {
#define CALL(X, W) return launch_gemm_t<X, W, false>(a, workspace, workspace_bytes, st)
  HQ_DISPATCH_FMT_PAIR(xf, wf, CALL);
#undef CALL
}

hipError_t launch_gemm_bsf(const GemmArgs& a, int xf, int wf, int bs, hipStream_t st) {
#define CALL(X, W)                                            \
  return bs == 32 ? launch_bsf_t<X, W, 32>(a, st)             \
         : bs == 64 ? launch_bsf_t<X, W, 64>(a, st) : launch_bsf_t<X, W, 128>(a, st)
  HQ_DISPATCH_FMT_PAIR(xf, wf, CALL);
#undef CALL
}

hipError_t launch_grouped_gemm(const GemmArgs& a, const int32_t* offsets, int experts, int xf, int wf,
                               hipStream_t st) {
#define CALL(X, W) return launch_grouped_t<X, W>(a, offsets, experts, st)
  HQ_DISPATCH_FMT_PAIR(xf, wf, CALL);
#undef CALL
}

}  // namespace hq
