// The a8w8 GEMM with bias, activation and residual in its epilogue, gfx950:
//
//   out[m, n] = act(x_scale[m] * w_scale[n] * sum_k dec(XQ[m,k]) * dec(WQ[n,k]) + bias[n]) + residual[m, n]
//
// on the plain GEMM's tiles and launch rules (gemm_kernels.h), with float32
// values up to the one rounding of the output.
#include "gemm_kernels.h"

namespace hq {

hipError_t launch_gemm_fused(const GemmArgs& a, int xf, int wf, void* workspace, size_t workspace_bytes, hipStream_t st) {
#define CALL(X, W) return launch_gemm_t<X, W, true>(a, workspace, workspace_bytes, st)
  HQ_DISPATCH_FMT_PAIR(xf, wf, CALL);
#undef CALL
}

}  // namespace hq
