// w4_fp8.cuh -- block-scaled 8-bit floating point (e4m3): quantization of
// weights (one fp32 scale per 128 x 128 block) and activations (one per token
// and 128 channels), and the residual RMS norm that writes its output in that
// form.
//
//   s = max|v over the block| / 448   (IEEE division; 1 if that is 0)
//   q = e4m3_rne(fp32(v / s))
//
// 448 is e4m3's largest value.  Where s is normal |v / s| <= 448 (1 + 2^-23),
// which rounds to 448; a subnormal s has few bits, the quotient can be up to 671,
// and the code saturates at 448.  The maximum is taken on the bit patterns of
// |v| as integers, whose order puts infinity and NaN above every finite value:
// a block that holds one gets the scale NaN and NaN codes, so a product with
// it is NaN instead of silently losing the value.
//
// The kernels start before the kernel ahead of them on the stream has ended
// (programmatic dependent launch).  What that kernel may write is read after
// the dependency wait and from L2 (ld.cg), every operand: this SM's L1 can still
// hold lines that the kernel before it read while this one was already
// resident, and a load declared read-only (ld.global.nc) may be moved ahead of
// the wait.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "w4_ptx.cuh"

namespace w4 {

constexpr int kFp8Block = 128;       // channels (and weight rows) per scale
constexpr float kFp8Max = 448.0f;    // largest e4m3 value

// A vector V at p, somewhere in an array of n elements from base: read from L2
// (zero where the bounds-checked build finds it outside), or written.
template <class V, class T>
__device__ __forceinline__ V ld_in(const T* p, const T* base, unsigned long long n) {
  if (!in_bounds(static_cast<unsigned long long>(p - base) + sizeof(V) / sizeof(T) - 1, n)) return V{};
  return __ldcg(reinterpret_cast<const V*>(p));
}
template <class T, class V>
__device__ __forceinline__ void st_in(T* p, const T* base, unsigned long long n, V v) {
  if (in_bounds(static_cast<unsigned long long>(p - base) + sizeof(V) / sizeof(T) - 1, n))
    *reinterpret_cast<V*>(p) = v;
}

// The scale of a block whose largest |v| has these bits.
__device__ __forceinline__ float fp8_scale(uint32_t max_bits) {
  if (max_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float s = __fdiv_rn(__uint_as_float(max_bits), kFp8Max);
  return s == 0.0f ? 1.0f : s;
}

// Two e4m3 codes, the first in the low byte (round to nearest even).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Scales along n channels or rows, for any n of an int.
__device__ __forceinline__ uint32_t fp8_blocks(int n) {
  return (static_cast<uint32_t>(n) + (kFp8Block - 1)) / kFp8Block;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// 8 bf16 values of a 16-byte load, widened.
__device__ __forceinline__ void unpack_bf16x8(uint4 w, float (&v)[8]) {
  const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(p[i] << 16);
    v[2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
  }
}

// Two floats as one operand of the two-wide fp32 instructions.
__device__ __forceinline__ unsigned long long f32x2(float lo, float hi) {
  unsigned long long d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ unsigned long long fma_f32x2(unsigned long long a, unsigned long long b,
                                                        unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long mul_f32x2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Codes of -u / s for 8 values u: two words.  An IEEE division per value costs
// more instructions than HBM speed leaves (about 16 per value at 3 bytes).
// The divisor is shared, so its reciprocal r, rounded to nearest, is taken
// once (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990: with such an r, and q within one ulp of v / s,
// q - r (q s - v) in two fused operations is the correctly rounded quotient).
// v r alone can be 1.5 ulp off, so a first step brings q within one ulp and
// the second rounds correctly.  This needs a normal r and no harmful underflow
// in q s - v: s >= 1e-25, and then a value so small that its remainder is
// inexact has the code 0 in any case.  With u = -v every step is one two-wide
// fma, q s + u and (q s + u) (-r) + q, and a zero keeps its sign.
__device__ __forceinline__ uint2 fp8_codes8_neg(const float (&u)[8], float s) {
  uint32_t c[4];
  if (s >= 1e-25f) {
    const float r = __frcp_rn(s);
    const unsigned long long s2 = f32x2(s, s), nr2 = f32x2(-r, -r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned long long u2 = f32x2(u[2 * i], u[2 * i + 1]);
      unsigned long long q = mul_f32x2(u2, nr2);
      q = fma_f32x2(fma_f32x2(q, s2, u2), nr2, q);
      q = fma_f32x2(fma_f32x2(q, s2, u2), nr2, q);
      float lo, hi;
      asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(q));
      c[i] = e4m3x2(lo, hi);
    }
  } else {  // tiny, or NaN
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3x2(__fdiv_rn(-u[2 * i], s), __fdiv_rn(-u[2 * i + 1], s));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// 8 bf16 values of a 16-byte load, widened and negated.
__device__ __forceinline__ void unpack_neg_bf16x8(uint4 w, float (&u)[8]) {
  constexpr uint32_t kSigns = 0x80008000u;
  unpack_bf16x8(make_uint4(w.x ^ kSigns, w.y ^ kSigns, w.z ^ kSigns, w.w ^ kSigns), u);
}

// Largest |v| bits over the 16 lanes of this half warp.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t a) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// Largest |v| of 8 bf16 values, as fp32 bits.  The magnitudes' patterns order
// as integers, two to a word.
__device__ __forceinline__ uint32_t abs_max_bf16x8(uint4 w) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & kMag, w.y & kMag), __vmaxu2(w.z & kMag, w.w & kMag));
  return max(m << 16, m & 0xFFFF0000u);
}

// ------------------------------------------------------------- activations
// Half a warp per (token, 128 channels): 8 channels per lane, one 16-byte
// load and one 8-byte store, U blocks in flight.  K % 16 == 0; with RAGGED the
// last block of a row is shorter (lanes past K hold nothing), without it the
// blocks are simply consecutive.  4099 x 13824 in 40 us, 4.3 TB/s.  Bound by
// instruction issue first: 17.5 instructions per value are 28 us of it (profile);
// then by the loads' latency, with 5 CTAs per SM (46 registers) and no load
// in flight while a turn's codes are made.  (One-wide fp32 arithmetic and U = 2
// 45 us, U = 1 53 us, U = 4 58 us.)
template <int U, bool RAGGED>
__global__ void __launch_bounds__(256)
    fp8_quantize_x_kernel(const uint16_t* X, long long blocks, int K, FastDivIdx by_kb, uint8_t* q,
                          float* s, unsigned long long values) {  // M K
  grid_dep_launch();
  grid_dep_wait();
  const int l = threadIdx.x & 15;
  const long long step = static_cast<long long>(gridDim.x) * 16;
  // every lane of a warp runs the same number of turns (the shuffles below)
  for (long long b0 = static_cast<long long>(blockIdx.x) * 16; b0 < blocks; b0 += U * step) {
    uint4 w[U];
    size_t at[U];
    bool have[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long b = b0 + u * step + threadIdx.x / 16;
      have[u] = b < blocks;
      at[u] = static_cast<size_t>(b) * kFp8Block + l * 8;
      if (RAGGED) {
        const uint32_t kb_n = fp8_blocks(K);
        const unsigned long long m = have[u] ? fast_div(static_cast<unsigned long long>(b), by_kb) : 0;
        const int k = static_cast<int>(b - static_cast<long long>(m * kb_n)) * kFp8Block + l * 8;
        have[u] = have[u] && k < K;
        at[u] = static_cast<size_t>(m) * K + k;
      }
      w[u] = have[u] ? ld_in<uint4>(X + at[u], X, values) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[8];  // negated
      unpack_neg_bf16x8(w[u], v);
      const float sc = fp8_scale(half_warp_max(abs_max_bf16x8(w[u])));
      if (have[u]) st_in(q + at[u], q, values, fp8_codes8_neg(v, sc));
      const long long b = b0 + u * step + threadIdx.x / 16;
      if (l == 0 && b < blocks) s[b] = sc;
    }
  }
}

// ----------------------------------------------------------------- weights
constexpr int kFp8WThreads = 256, kFp8WBlocks = 3;

// One CTA per 128 x 128 block of one of B matrices: 16 lanes per row, 8
// channels per lane, 16 rows at a time; the values stay in registers between
// the maximum and the codes.  Bound by HBM: 16 x 2000 x 4096 in 106 us, 6.2 TB/s;
// a single matrix of 4096 x 4096, 17 us, by 1024 CTAs on 444 places.  Three CTAs
// per SM leave 80 registers, 28 bytes short (they spill to the stack); 2 CTAs
// per SM, or CTAs of 512 threads, 2 per SM, were slower by 10 % and 3 %.
__global__ void __launch_bounds__(kFp8WThreads, kFp8WBlocks)
    fp8_quantize_w_kernel(const float* W, int N, int K, uint8_t* q, float* s,
                          unsigned long long values) {  // B N K
  constexpr int kRows = kFp8WThreads / 16, kTurns = kFp8Block / kRows;
  __shared__ uint32_t wmax[kFp8WThreads / 32];
  const uint32_t kb_n = fp8_blocks(K), nb_n = fp8_blocks(N);
  const uint32_t bn = blockIdx.x / kb_n, kb = blockIdx.x - bn * kb_n;
  const uint32_t mat = bn / nb_n;
  const int nb = static_cast<int>(bn - mat * nb_n);
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int k = static_cast<int>(kb) * kFp8Block + l * 8;
  const float* Wm = W + static_cast<size_t>(mat) * N * K;
  float v[kTurns][8];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int n = nb * kFp8Block + r0 + kRows * i;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (n < N && k < K &&
        in_bounds(static_cast<unsigned long long>(Wm - W) + static_cast<size_t>(n) * K + k + 7, values)) {
      const float4* p = reinterpret_cast<const float4*>(Wm + static_cast<size_t>(n) * K + k);
      a = __ldcs(p);
      b = __ldcs(p + 1);
    }
    v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
    v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = max(mx, abs_bits(v[i][j]));
  }
  mx = half_warp_max(mx);
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = wmax[0];
#pragma unroll
  for (int i = 1; i < kFp8WThreads / 32; ++i) mx = max(mx, wmax[i]);
  const float sc = fp8_scale(mx);
  uint8_t* qm = q + static_cast<size_t>(mat) * N * K;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int n = nb * kFp8Block + r0 + kRows * i;
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = -v[i][j];
    if (n < N && k < K) st_in(qm + static_cast<size_t>(n) * K + k, q, values, fp8_codes8_neg(u, sc));
  }
  if (threadIdx.x == 0) s[blockIdx.x] = sc;
}

// ---------------------------------------------------------------- RMS norm
// One CTA per token: r = x + residual in fp32 (kept in registers, 8 channels
// per chunk, CPT chunks per thread), the mean of r^2 over the CTA, then
// y = r * rsqrt(mean + eps) * w in fp32 and its codes without a rounding in
// between.  residual_out is bf16(r); the norm itself uses the unrounded sum.
// Every thread reads its own channels before it writes them, so residual_out
// may be residual or x.  Bound by HBM: 8191 x 8192 with every output in 100 to
// 106 us, 5.7 to 6.1 TB/s; one row of 4096 in 2.4 us, the launch.  Above 32768
// channels a thread's 64 values spill in part (224 bytes).
// Up to 16384 channels a thread has 32 registers, which fills an SM with threads;
// left to itself the compiler's choice moves with small changes (50 registers:
// 8191 x 8192 in 129 us).
template <int CPT>
__global__ void __launch_bounds__(1024, CPT <= 2 ? 2 : 1) fp8_add_rmsnorm_kernel(
    const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
    int K, uint16_t* residual_out, uint16_t* y_out, uint8_t* q, float* s) {
  __shared__ float part[32];
  grid_dep_launch();
  grid_dep_wait();
  const size_t row = static_cast<size_t>(blockIdx.x) * K;
  const unsigned long long values = static_cast<unsigned long long>(gridDim.x) * K;
  float v[CPT][8];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int k = (static_cast<int>(threadIdx.x) + c * static_cast<int>(blockDim.x)) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
    if (k < K) {
      unpack_bf16x8(ld_in<uint4>(x + row + k, x, values), v[c]);
      if (residual) {
        float r[8];
        unpack_bf16x8(ld_in<uint4>(residual + row + k, residual, values), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] += r[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[c][j], v[c][j], ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  float total = 0.0f;
  for (int w = 0; w < warps; ++w) total += part[w];
  const float rstd = rsqrtf(total / static_cast<float>(K) + eps);
  const int kb_n = (K + kFp8Block - 1) / kFp8Block;  // K <= 65536
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int k = (static_cast<int>(threadIdx.x) + c * static_cast<int>(blockDim.x)) * 8;
    const bool have = k < K;
    if (have && residual_out) {
      uint4 o;
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[j] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[c][2 * j]))) |
               (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[c][2 * j + 1]))) << 16);
      o.x = p[0]; o.y = p[1]; o.z = p[2]; o.w = p[3];
      st_in(residual_out + row + k, residual_out, values, o);
    }
    float w8[8] = {};
    if (have) unpack_bf16x8(ld_in<uint4>(weight + k, weight, K), w8);
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[c][j] = v[c][j] * -rstd * w8[j];  // -y
      mx = max(mx, abs_bits(v[c][j]));
    }
    if (!have) mx = 0;  // 0 * rstd is NaN where rstd is not finite
    mx = half_warp_max(mx);
    if (!have) continue;
    const float sc = fp8_scale(mx);
    if (y_out) {
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[j] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(-v[c][2 * j]))) |
               (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(-v[c][2 * j + 1]))) << 16);
      st_in(y_out + row + k, y_out, values, make_uint4(p[0], p[1], p[2], p[3]));
    }
    st_in(q + row + k, q, values, fp8_codes8_neg(v[c], sc));
    if ((threadIdx.x & 15) == 0 && in_bounds(k / kFp8Block, kb_n))
      s[static_cast<size_t>(blockIdx.x) * kb_n + k / kFp8Block] = sc;
  }
}

}  // namespace w4
