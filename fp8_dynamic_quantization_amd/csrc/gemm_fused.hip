// The a8w8 GEMM with bias, activation and residual in its epilogue, gfx950:
//
//   out[m, n] = act(x_scale[m] * w_scale[n] * sum_k dec(XQ[m,k]) * dec(WQ[n,k]) + bias[n]) + residual[m, n]
//
// on the plain GEMM's tiles and launch rules (gemm_kernels.h), with float32
// values up to the one rounding of the output. Large shapes are bound by the K loop: on
// one card, replayed from graphs, 4096 x 4096 x 4096 takes 52.3 us in the plain form,
// 55.5 here without activation and residual (the same bits as the epilogue form), 58.7
// with the residual and 61.8 (2.2 PFLOP/s) with tanh-GELU and residual.
#include "gemm_kernels.h"

namespace hq {

// ---------------------------------------------------------------------------
// 17 to 64 rows: one barrier
// ---------------------------------------------------------------------------
// A decode batch of more than one 16-row block is bound by latency: the weight is
// read once (14.7 MB at N = 7168, K = 2048: 2.4 us at 6.15 TB/s; 33 rows take 6.1 to
// 6.7, one row in the weight-streaming kernel 4.3 to 4.8), but a wavefront that walks
// over several chunks of K pays a round trip for each, and adding every slice's
// sums across wavefronts one after the other costs two barriers a slice. Here a
// workgroup owns F weight fragments (16 F columns) and all rows, its W wavefronts
// take the K blocks w, w + W, ... two at a time, every sum goes to LDS at once,
// and after one barrier wavefront w adds slice w of the F * MB slices in wavefront
// order and runs its epilogue.
template <int XF, int WF, int MB, int F, int W>
__global__ __launch_bounds__(64 * W) void gemm_rows_kernel(GemmArgs a) {
  constexpr int KPW = 2;
  constexpr int S = F * MB;  // slices
  __shared__ __attribute__((aligned(16))) v4f red[W][S][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = a.k, nkb = (K + kBK - 1) / kBK;
  const int nfrag = frag_rows(a.n);
  const int nb0 = blockIdx.x * F;
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.wq_pre + (size_t)nb0 * nkb * kFragBytes), (short)0, min(F, nfrag - nb0) * nkb * kFragBytes, kRsrcFlags);
  const __amdgpu_buffer_rsrc_t x_rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)a.xq, (short)0, a.m * K, kRsrcFlags);
  const int xr = lane & 15, xc = 32 * (lane >> 4);

  v4f acc[F][MB];
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[f][i] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb0 = wave; kb0 < nkb; kb0 += KPW * W) {
    uint4 fb[KPW][F][2], fx[KPW][MB][2];
#pragma unroll
    for (int j = 0; j < KPW; ++j) {
      const int kb = kb0 + j * W;
      const int bvo = kb < nkb ? lane * 16 : kBadOffset;  // past nkb lies the next fragment's row
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          fb[j][f][h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(b_rsrc, bvo + h * 1024,
                                                                       (f * nkb + min(kb, nkb - 1)) * kFragBytes, kNtLoad));
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = kb * kBK + xc + 16 * h;
          fx[j][i][h] = as_uint4(__builtin_amdgcn_raw_buffer_load_b128(x_rsrc, col < K ? (i * 16 + xr) * K + col : kBadOffset, 0, 0));
        }
    }
    __builtin_amdgcn_sched_barrier(0);  // every load of the chunk ahead of its first MFMA
#pragma unroll
    for (int j = 0; j < KPW; ++j)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const uint4 &b0 = fb[j][f][0], &b1 = fb[j][f][1];
        const v8i bw = v8i{(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const uint4 &x0 = fx[j][i][0], &x1 = fx[j][i][1];
          const v8i xa = v8i{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
          acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bw, xa, acc[f][i], WF, XF, 0, 0, 0, 0);
        }
      }
  }

  // The slice this wavefront finishes: its scales, bias and residual are fetched
  // while the sums go through LDS. Lane l holds row 16 i + l % 16 and 4 columns.
  const int sl = wave;
  const int f = sl / MB, i = sl % MB, nb = nb0 + f;
  const int row = i * 16 + xr, col0 = 32 * (nb >> 1) + 8 * (lane >> 4) + 4 * (nb & 1);
  const bool mine = sl < S && row < a.m && col0 < a.n;
  float xsc = 0.0f, wsc[4] = {}, bias[4] = {};
  uint4 res = make_uint4(0u, 0u, 0u, 0u);
  if (mine) {
    xsc = a.x_scale[a.x_scale_per_row ? row : 0];
    const float bsc = a.bias_kind > kBiasBF16 ? a.bias_scale[0] : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = min(col0 + e, a.n - 1);
      wsc[e] = a.w_scale[a.w_scale_per_col ? col : 0];
      if (a.bias_kind != kBiasNone) bias[e] = bias_at(a, col, bsc);
    }
    if (a.residual) res = residual4(a, row, col0);
  }
#pragma unroll
  for (int q = 0; q < S; ++q) red[wave][q][lane] = acc[q / MB][q % MB];
  __syncthreads();
  if (!mine) return;
  v4f t = red[0][sl][lane];
#pragma unroll
  for (int w = 1; w < W; ++w) t += red[w][sl][lane];
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = t[e] * xsc * wsc[e];
  if (a.bias_kind != kBiasNone) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += bias[e];
  }
  fused_values<4>(a, v, res);
  const size_t off = (size_t)row * a.n + col0;
  const bool full = (a.n & 3) == 0;
  if (a.out_scale) {
    store_fp8_out<4>(static_cast<uint8_t*>(a.out) + off, v, 1.0f / a.out_scale[0], a.out_fmt, full, a.n - col0);
    return;
  }
  const uint32_t w0 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[0], v[1]}), bf2v));
  const uint32_t w1 = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[2], v[3]}), bf2v));
  uint16_t* dst = static_cast<uint16_t*>(a.out) + off;
  if (full) {
    __builtin_nontemporal_store(hq_u2v{w0, w1}, reinterpret_cast<hq_u2v*>(dst));
  } else {
    for (int e = 0; e < 4; ++e)
      if (col0 + e < a.n) dst[e] = (uint16_t)((e < 2 ? w0 : w1) >> (16 * (e & 1)));
  }
}

// One fragment per workgroup while that gives every CU at most one, else two: two
// halve the rereading of X from the L2 but leave CUs idle below 512 fragments.
// Measured (us, one / two): N = 7168, K = 2048, M = 33 8.2 / 6.5; N = 4096, K = 4096,
// M = 64 11.3 / 12.2; N = 512, K = 8192, M = 20 9.0 / 10.9. Sixteen wavefronts were
// slower on the wide shapes (8.5 -> 15.8 at N = 7168, K = 2048, M = 64) and within 4 %
// on the narrow ones. The weight-streaming kernel takes 12.6, 15.5 and 12.3 us.
template <int XF, int WF, int MB>
static hipError_t launch_rows(const GemmArgs& a, hipStream_t st) {
  const int nfrag = frag_rows(a.n);
  if (nfrag <= kNumCUs)
    hipLaunchKernelGGL((gemm_rows_kernel<XF, WF, MB, 1, 8>), dim3(nfrag), dim3(512), 0, st, a);
  else
    hipLaunchKernelGGL((gemm_rows_kernel<XF, WF, MB, 2, 8>), dim3((nfrag + 1) / 2), dim3(512), 0, st, a);
  return hipGetLastError();
}

template <int XF, int WF>
static hipError_t launch_fused_t(const GemmArgs& a, void* workspace, size_t workspace_bytes, hipStream_t st) {
  if (a.m > 16 && a.m <= kSkinnyMaxM) {
    if (a.m <= 32) return launch_rows<XF, WF, 2>(a, st);
    if (a.m <= 48) return launch_rows<XF, WF, 3>(a, st);
    return launch_rows<XF, WF, 4>(a, st);
  }
  return launch_gemm_t<XF, WF, true>(a, workspace, workspace_bytes, st);
}

hipError_t launch_gemm_fused(const GemmArgs& a, int xf, int wf, void* workspace, size_t workspace_bytes, hipStream_t st) {
#define CALL(X, W) return launch_fused_t<X, W>(a, workspace, workspace_bytes, st)
  HQ_DISPATCH_FMT_PAIR(xf, wf, CALL);
#undef CALL
}

}  // namespace hq
