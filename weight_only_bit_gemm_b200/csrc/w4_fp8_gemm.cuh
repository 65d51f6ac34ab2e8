// w4_fp8_gemm.cuh -- Y[m,n] = sum over 128-channel blocks j of
//   sx[m,j] * sw[n/128,j] * sum over k in j of qx[m,k] * qw[n,k]
// for e4m3 codes (the product of two codes is exact in fp32).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "w4_fp8.cuh"

namespace w4 {

struct Fp8GemmArgs {
  const uint8_t* qx;  // [M, K]
  const float* sx;    // [M, KB]
  const uint8_t* qw;  // [N, K]
  const float* sw;    // [ceil(N / 128), KB]
  uint16_t* Y;        // bf16 [M, N]
  int M, N, K, KB;
};

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

// 64 x 64 outputs per CTA, 4 x 4 per thread, one 128-channel block at a time.
__global__ void __launch_bounds__(256) fp8_gemm_simple_kernel(const Fp8GemmArgs a) {
  __shared__ float xs[64][33], wsm[64][33];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int kb = 0; kb < a.KB; ++kb) {
    float part[4][4] = {};
    for (int k0 = kb * kFp8Block; k0 < min(a.K, (kb + 1) * kFp8Block); k0 += 32) {
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int r = i >> 5, k = k0 + (i & 31);
        xs[r][i & 31] = m0 + r < a.M && k < a.K ? e4m3_f32(a.qx[static_cast<size_t>(m0 + r) * a.K + k]) : 0.f;
        wsm[r][i & 31] = n0 + r < a.N && k < a.K ? e4m3_f32(a.qw[static_cast<size_t>(n0 + r) * a.K + k]) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            part[i][j] = fmaf(xs[ty + 16 * i][k], wsm[tx + 16 * j][k], part[i][j]);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < a.M && n < a.N)
          acc[i][j] = fmaf(part[i][j],
                           a.sx[static_cast<size_t>(m) * a.KB + kb] *
                               a.sw[static_cast<size_t>(n / kFp8Block) * a.KB + kb],
                           acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N)
        a.Y[static_cast<size_t>(m) * a.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i][j]));
    }
}

}  // namespace w4
