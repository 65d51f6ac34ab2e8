// w4_fp8_moe.cuh -- a mixture-of-experts layer over block-scaled e4m3 experts
// for a few tokens: routing, gate and up products, SiLU, down product and the
// weighted sum.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "w4_fp8_gemm.cuh"

namespace w4 {

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

constexpr int kMoeMaxTokens = 128;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTop = 16;

struct MoeArgs {
  const uint16_t* X;       // bf16 [T, H]
  const uint16_t* router;  // bf16 [E, H]
  const uint8_t* w13;      // [E, 2, I, H]: gate, up
  const float* s13;        // [E, 2, IB, HB]
  const uint8_t* w2;       // [E, H, I]
  const float* s2;         // [E, HB, IB]
  uint16_t* Y;             // bf16 [T, H]
  int32_t* ids;            // [T, top]
  float* weights;          // [T, top]
  uint8_t* xq;             // [T, H]
  float* sx;               // [T, HB]
  float* h;                // [T * top, I]
  uint8_t* hq;             // [T * top, I]
  float* sh;               // [T * top, IB]
  int T, E, top, H, I, HB, IB, renorm;
};

// A logit's place in the order of the choice: NaN below every number.
__device__ __forceinline__ float moe_key(float v) { return v == v ? v : -INFINITY; }

// One CTA per token: logits (a warp per expert), the `top` largest (ties: the
// lowest index), their softmax weights, and the token's e4m3 codes.
__global__ void __launch_bounds__(256) moe_route_simple_kernel(const MoeArgs a) {
  __shared__ float logit[kMoeMaxExperts];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint16_t* x = a.X + static_cast<size_t>(t) * a.H;
  for (int e = warp; e < a.E; e += 8) {
    const uint16_t* r = a.router + static_cast<size_t>(e) * a.H;
    float d = 0.0f;
    for (int k = lane; k < a.H; k += 32)
      d = fmaf(__uint_as_float(static_cast<uint32_t>(x[k]) << 16),
               __uint_as_float(static_cast<uint32_t>(r[k]) << 16), d);
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) logit[e] = d;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float lmax = 0.0f, all = 0.0f, chosen = 0.0f;
    for (int j = 0; j < a.top; ++j) {
      int best = -1;
      for (int e = 0; e < a.E; ++e) {
        bool used = false;
        for (int i = 0; i < j; ++i) used |= a.ids[t * a.top + i] == e;
        if (!used && (best < 0 || moe_key(logit[e]) > moe_key(logit[best]))) best = e;
      }
      if (j == 0) lmax = logit[best];
      a.ids[t * a.top + j] = best;
      chosen += expf(logit[best] - lmax);
    }
    for (int e = 0; e < a.E; ++e) all += expf(logit[e] - lmax);
    for (int j = 0; j < a.top; ++j)
      a.weights[t * a.top + j] =
          expf(logit[a.ids[t * a.top + j]] - lmax) / (a.renorm ? chosen : all);
  }
}

// h = silu(gate) * up for one (token, choice): a warp per channel.
__global__ void __launch_bounds__(256) moe_up_simple_kernel(const MoeArgs a) {
  const int p = blockIdx.x, t = p / a.top, lane = threadIdx.x & 31;
  const int e = a.ids[p];
  const int i = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (i >= a.I) return;
  float gu[2] = {0.0f, 0.0f};
  for (int kb = 0; kb < a.HB; ++kb) {
    float d[2] = {0.0f, 0.0f};
    for (int k = kb * 128 + lane; k < min(a.H, kb * 128 + 128); k += 32) {
      const float xv = e4m3_f32(a.xq[static_cast<size_t>(t) * a.H + k]);
      for (int g = 0; g < 2; ++g)
        d[g] = fmaf(xv, e4m3_f32(a.w13[((static_cast<size_t>(e) * 2 + g) * a.I + i) * a.H + k]), d[g]);
    }
    for (int g = 0; g < 2; ++g) {
      for (int o = 16; o > 0; o >>= 1) d[g] += __shfl_xor_sync(0xffffffffu, d[g], o);
      gu[g] = fmaf(d[g], a.sx[t * a.HB + kb] *
                             a.s13[((static_cast<size_t>(e) * 2 + g) * a.IB + i / 128) * a.HB + kb], gu[g]);
    }
  }
  if (lane == 0) a.h[static_cast<size_t>(p) * a.I + i] = gu[0] / (1.0f + expf(-gu[0])) * gu[1];
}

// Codes of h: a CTA of 128 threads per (row, block).
__global__ void __launch_bounds__(128) moe_quantize_h_kernel(const MoeArgs a) {
  __shared__ uint32_t mx[4];
  const int p = blockIdx.x, ib = blockIdx.y, i = ib * 128 + threadIdx.x;
  const float v = i < a.I ? a.h[static_cast<size_t>(p) * a.I + i] : 0.0f;
  uint32_t m = abs_bits(v);
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) mx[threadIdx.x >> 5] = m;
  __syncthreads();
  const float s = fp8_scale(max(max(mx[0], mx[1]), max(mx[2], mx[3])));
  if (i < a.I) a.hq[static_cast<size_t>(p) * a.I + i] = static_cast<uint8_t>(e4m3x2(__fdiv_rn(v, s), 0.0f));
  if (threadIdx.x == 0) a.sh[p * a.IB + ib] = s;
}

// y[t, n]: a warp per (token, channel), the choices in order.
__global__ void __launch_bounds__(256) moe_down_simple_kernel(const MoeArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int n = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (n >= a.H) return;
  float y = 0.0f;
  for (int j = 0; j < a.top; ++j) {
    const int p = t * a.top + j, e = a.ids[p];
    float acc = 0.0f;
    for (int kb = 0; kb < a.IB; ++kb) {
      float d = 0.0f;
      for (int k = kb * 128 + lane; k < min(a.I, kb * 128 + 128); k += 32)
        d = fmaf(e4m3_f32(a.hq[static_cast<size_t>(p) * a.I + k]),
                 e4m3_f32(a.w2[(static_cast<size_t>(e) * a.H + n) * a.I + k]), d);
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      acc = fmaf(d, a.sh[p * a.IB + kb] * a.s2[(static_cast<size_t>(e) * a.HB + n / 128) * a.IB + kb], acc);
    }
    y = fmaf(a.weights[p], acc, y);
  }
  if (lane == 0) a.Y[static_cast<size_t>(t) * a.H + n] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

}  // namespace w4
