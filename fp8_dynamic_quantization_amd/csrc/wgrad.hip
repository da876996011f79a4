// Weight gradient from the FP8 codes that the forward GEMM read, gfx950:
//
//   dW[n, k] = base[n, k] + sum_m G[m, n] * x_scale[m] * dec(XQ[m, k])
//
// G bf16 [m, n], XQ uint8 [m, k], both row-major, so the contraction runs over
// the slow axis of both.
#include "hq_launch.h"
#include "hq_row.h"

namespace hq {

// A 64 x 64 tile per workgroup, 4 x 4 outputs per thread, 16 tokens staged in
// LDS at a time as float32.
template <int XF>
__global__ __launch_bounds__(256) void wgrad_kernel(WgradArgs a) {
  __shared__ float sg[16][64], sx[16][64];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * 64, k0 = (int64_t)blockIdx.x * 64;
  float acc[4][4] = {};
  for (int64_t m0 = 0; m0 < a.m; m0 += 16) {
    for (int i = tid; i < 1024; i += 256) {
      const int r = i >> 6, c = i & 63;
      const int64_t m = m0 + r;
      float g = 0.0f, x = 0.0f;
      if (m < a.m) {
        if (n0 + c < a.n) g = __uint_as_float((uint32_t)a.g[(size_t)m * a.n + n0 + c] << 16) * a.x_scale[a.x_scale_per_row ? m : 0];
        if (k0 + c < a.k) {
          const int code = a.xq[(size_t)m * a.k + k0 + c];
          x = XF == kE4M3 ? __builtin_amdgcn_cvt_f32_fp8(code, 0) : __builtin_amdgcn_cvt_f32_bf8(code, 0);
        }
      }
      sg[r][c] = g;
      sx[r][c] = x;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sg[r][ty * 4 + i], sx[r][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + ty * 4 + i, k = k0 + tx * 4 + j;
      if (n >= a.n || k >= a.k) continue;
      const size_t at = (size_t)n * a.k + k;
      const float v = a.base ? acc[i][j] + a.base[at] : acc[i][j];
      if (a.out_f32) static_cast<float*>(a.dw)[at] = v;
      else static_cast<uint16_t*>(a.dw)[at] = (uint16_t)f32_to_bf16_rne(v);
    }
}

size_t wgrad_workspace_bytes(int, int, int, bool) { return 0; }

hipError_t launch_wgrad(const WgradArgs& a, int xf, void*, size_t, hipStream_t st) {
  const dim3 grid((a.k + 63) / 64, (a.n + 63) / 64);
  if (xf == kE4M3) hipLaunchKernelGGL(wgrad_kernel<kE4M3>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(wgrad_kernel<kE5M2>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace hq
