// w4_fp8_moe.cuh -- a mixture-of-experts layer over block-scaled e4m3 experts
// for up to 128 tokens, in two kernels:
//
//   moe_route_kernel   router logits, the choice of experts and their weights,
//                      the tokens' e4m3 codes, the list of active experts;
//   moe_expert_kernel  gate and up products with SiLU and the codes of h, then
//                      the down products with the weighted sum.
//
// With few tokens the layer reads every active expert's weights once and is
// bound by that stream, so each weight tile meets all the tokens: they are the
// MMA's 128 rows as in fp8_rows_gemm_kernel, and a token that did not choose
// the expert is a lane whose sums are left out.  Nothing is gathered or sorted;
// h has a row for every (active expert, token), of which the chosen ones are
// written and used.
//
// The down product's weight is linear in the block sums, so a cluster runs over
// the blocks of all active experts in one pass with the routing weight folded
// into the block's scale, and an output is written once.
//
// The expert kernel's clusters take their work by a counter, the gate and up
// part first.  A cluster that waits for h therefore waits for clusters that
// already run, whatever else occupies the GPU.
#pragma once

#include "w4_fp8_gemm.cuh"

namespace w4 {

constexpr int kMoeMaxTokens = 128;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTop = 16;
constexpr int kMoeCluster = 8;       // CTAs of an expert-kernel cluster
constexpr int kMoeRouteTokens = 4;   // tokens per routing CTA
constexpr int kMoeRouteExperts = 8;  // experts per routing CTA (a warp each)

// Counters of a call, all zero between calls.
struct MoeCounters {
  unsigned int ticket;     // expert-kernel clusters started
  unsigned int h_done;     // CTAs that have published their part of h
  unsigned int left;       // expert-kernel clusters finished
  unsigned int groups;     // token groups routed
  unsigned int group[kMoeMaxTokens / kMoeRouteTokens];  // routing CTAs done per group
};

struct MoeArgs {
  const uint16_t* X;       // bf16 [T, H]
  const uint16_t* router;  // bf16 [E, H]
  const float* s13;        // [E, 2, IB, HB]
  const float* s2;         // [E, HB, IB]
  uint16_t* Y;             // bf16 [T, H]
  int32_t* ids;            // [T, top]
  float* weights;          // [T, top]
  uint8_t* xq;             // [T, H]
  float* sx;               // [T, HB]
  float* logits;           // [T, E]
  int32_t* active;         // [0] their number, then their experts, ascending
  float* wt;               // [A, T]: routing weight, -1 where the token did not choose the expert
  uint8_t* hq;             // [A, T, I]
  float* sh;               // [A, T, IB]
  MoeCounters* cnt;
  int T, E, top, H, I, HB, IB, renorm;
  int A;                   // most experts that can be active
  int route_ctas;          // routing CTAs; the ones after them quantize X
  int ksplit;              // K ranges of a gate and up tile
  int vec;                 // Y rows are 8-byte aligned
  int vec13, vec2;         // rows of s13 and sx, of s2 and sh, are 16-byte aligned
};

// ------------------------------------------------------------------ routing
// Order of the choice: larger logits first, NaN below every number, as an
// unsigned key that is never 0.
__device__ __forceinline__ uint32_t moe_key(float v) {
  const uint32_t b = __float_as_uint(v == v ? v + 0.0f : -INFINITY);  // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A CTA of 8 warps: 8 experts (one per warp) x 4 tokens of logits; the last CTA
// of a token group chooses its experts, and the last group's CTA lists the
// active ones.  The CTAs after route_ctas write the tokens' codes.
__global__ void __launch_bounds__(256) moe_route_kernel(const MoeArgs a) {
  __shared__ uint32_t flags[kMoeMaxExperts];
  __shared__ int slot[kMoeMaxExperts];
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  grid_dep_wait();

  if (static_cast<int>(blockIdx.x) >= a.route_ctas) {
    // 16 lanes per (token, 128 channels)
    const int b = (static_cast<int>(blockIdx.x) - a.route_ctas) * 16 + (threadIdx.x >> 4);
    const int l = threadIdx.x & 15;
    const bool live = b < a.T * a.HB;
    const int m = live ? b / a.HB : 0, k = (b - m * a.HB) * kFp8Block + l * 8;
    const bool have = live && k < a.H;
    const size_t at = static_cast<size_t>(m) * a.H + k;
    const unsigned long long n_x = static_cast<unsigned long long>(a.T) * a.H;
    const uint4 w = have ? ld_in<uint4>(a.X + at, a.X, n_x) : make_uint4(0u, 0u, 0u, 0u);
    float v[8];  // negated
    unpack_neg_bf16x8(w, v);
    const float sc = fp8_scale(half_warp_max(abs_max_bf16x8(w)));
    if (have) st_in(a.xq + at, a.xq, n_x, fp8_codes8_neg(v, sc));
    if (live && l == 0) st_in(a.sx + b, a.sx, static_cast<unsigned long long>(a.T) * a.HB, sc);
    return;
  }

  const int eg = (a.E + kMoeRouteExperts - 1) / kMoeRouteExperts;  // CTAs of a token group
  const int tg = static_cast<int>(blockIdx.x) / eg;
  const int t0 = tg * kMoeRouteTokens;
  const int e = (static_cast<int>(blockIdx.x) - tg * eg) * kMoeRouteExperts + warp;
  if (e < a.E) {
    float d[kMoeRouteTokens] = {};
    const uint16_t* r = a.router + static_cast<size_t>(e) * a.H;
    const int tokens = min(kMoeRouteTokens, a.T - t0);
    const uint16_t* x = a.X + static_cast<size_t>(t0) * a.H;
    // 8 chunks of the expert's row in flight, then the tokens' one by one
    for (int k = lane * 8; k < a.H; k += 8 * 256) {
      uint4 rw[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        rw[c] = k + c * 256 < a.H ? ld_in<uint4>(r + k + c * 256, a.router,
                                                 static_cast<unsigned long long>(a.E) * a.H)
                                  : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < kMoeRouteTokens; ++i) {
        if (i >= tokens) break;
        uint4 xw[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          xw[c] = k + c * 256 < a.H
                      ? ld_in<uint4>(x + static_cast<size_t>(i) * a.H + k + c * 256, a.X,
                                     static_cast<unsigned long long>(a.T) * a.H)
                      : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float rv[8], xv[8];
          unpack_bf16x8(rw[c], rv);
          unpack_bf16x8(xw[c], xv);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[i] = fmaf(rv[j], xv[j], d[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kMoeRouteTokens; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d[i] += __shfl_xor_sync(0xffffffffu, d[i], o);
      if (lane == 0 && t0 + i < a.T)
        st_in(a.logits + static_cast<size_t>(t0 + i) * a.E + e, a.logits,
              static_cast<unsigned long long>(a.T) * a.E, d[i]);
    }
  }
  // (the barrier and thread 0's acquire-release publish the CTA's logits and
  // make the other CTAs' visible)
  __syncthreads();
  if (threadIdx.x == 0) {
    last = eg == 1 || (in_bounds(tg, kMoeMaxTokens / kMoeRouteTokens) &&
                       atom_add_acq_rel_gpu(&a.cnt->group[tg], 1u) == static_cast<unsigned>(eg - 1))
               ? 1 : 0;
    if (last && eg > 1) a.cnt->group[tg] = 0u;
  }
  __syncthreads();
  if (!last) return;

  // this group's logits are complete: a warp per token, E / 32 keys per lane
  constexpr int kPer = kMoeMaxExperts / 32;
  const int t = t0 + warp;
  if (warp < kMoeRouteTokens && t < a.T) {
    float v[kPer];
    uint32_t key[kPer];
    float lmax = 0.0f, mine = 0.0f, chosen = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = i * 32 + lane;
      v[i] = x < a.E ? ld_in<float>(a.logits + static_cast<size_t>(t) * a.E + x, a.logits,
                                    static_cast<unsigned long long>(a.T) * a.E)
                     : 0.0f;
      key[i] = x < a.E ? moe_key(v[i]) : 0u;
    }
    int pick = 0;       // lane j keeps choice j
    float weight = 0.0f;
    for (int j = 0; j < a.top; ++j) {
      uint32_t best = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i * 32 >= a.E) break;
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
      }
      const uint32_t top_key = __reduce_max_sync(0xffffffffu, best);
      const int e_best = static_cast<int>(__reduce_min_sync(
          0xffffffffu, best == top_key ? static_cast<uint32_t>(at * 32 + lane) : 0xffffffffu));
      float lv = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i * 32 >= a.E) break;
        if (i * 32 + lane == e_best) {
          key[i] = 0u;
          lv = v[i];
        }
      }
      lv = __shfl_sync(0xffffffffu, lv, e_best & 31);
      if (j == 0) lmax = lv;
      const float ex = expf(lv - lmax);
      chosen += ex;
      if (lane == j) {
        pick = e_best;
        weight = ex;
      }
    }
    float total = chosen;
    if (!a.renorm) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i * 32 >= a.E) break;
        if (i * 32 + lane < a.E) mine += expf(v[i] - lmax);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
      total = mine;
    }
    if (lane < a.top) {
      st_in(a.ids + t * a.top + lane, a.ids, static_cast<unsigned>(a.T * a.top), pick);
      st_in(a.weights + t * a.top + lane, a.weights, static_cast<unsigned>(a.T * a.top), weight / total);
    }
  }
  __syncthreads();
  const int ng = (a.T + kMoeRouteTokens - 1) / kMoeRouteTokens;
  if (ng > 1) {
    if (threadIdx.x == 0) {
      last = atom_add_acq_rel_gpu(&a.cnt->groups, 1u) == static_cast<unsigned>(ng - 1) ? 1 : 0;
      if (last) a.cnt->groups = 0u;
    }
    __syncthreads();
    if (!last) return;
  }

  // every token is routed: the active experts in ascending order, and each
  // one's weights by token
  for (int i = threadIdx.x; i < a.E; i += 256) flags[i] = 0u;
  __syncthreads();
  const int pairs = a.T * a.top;
  for (int i = threadIdx.x; i < pairs; i += 256) {
    const int e = __ldcg(a.ids + i);
    if (in_bounds(e, a.E)) flags[e] = 1u;
  }
  __syncthreads();
  if (warp == 0) {
    int base = 0;
    for (int i = 0; i < a.E; i += 32) {
      const bool on = i + lane < a.E && flags[i + lane] != 0u;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      const int at = base + __popc(m & ((1u << lane) - 1u));
      if (on && in_bounds(at, a.A)) {
        slot[i + lane] = at;
        a.active[1 + at] = i + lane;
      }
      base += __popc(m);
    }
    if (lane == 0) {
      a.active[0] = base;
      last = base;
    }
  }
  __syncthreads();
  const unsigned n_wt = static_cast<unsigned>(a.A * a.T);
  for (int i = threadIdx.x; i < last * a.T; i += 256) st_in(a.wt + i, a.wt, n_wt, -1.0f);
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += 256) {
    const int e = __ldcg(a.ids + i);
    if (in_bounds(e, a.E))
      st_in(a.wt + static_cast<size_t>(slot[e]) * a.T + i / a.top, a.wt, n_wt, __ldcg(a.weights + i));
  }
}

// ------------------------------------------------------------------ experts
__device__ __forceinline__ unsigned ld_acquire_gpu(const unsigned int* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Add without waiting for the old value; publishes this thread's earlier writes
// and, through a barrier before it, those of its CTA.
__device__ __forceinline__ void red_add_release_gpu(unsigned int* p, unsigned int v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// The expert of active slot i.
__device__ __forceinline__ int moe_expert(const MoeArgs& a, int i) {
  const int e = ld_in<int>(a.active + 1 + i, a.active, a.A + 1);
  return in_bounds(e, a.E) ? e : 0;
}

// Bounded wait until a counter in global memory has reached `want`.
__device__ __forceinline__ bool wait_counter(const unsigned int* counter, unsigned want,
                                             long long limit = kWaitLimitCycles) {
  const long long t0 = clock64();
  while (ld_acquire_gpu(counter) < want) {
    if (clock64() - t0 > limit) {
      set_dev_error(W4_DEV_ERR_TIMEOUT);
      return false;
    }
    __nanosleep(64);
  }
  return true;
}
// ... until every gate and up CTA has published its part of h.
__device__ __forceinline__ bool moe_wait_h(const MoeArgs& a, unsigned want) {
  return wait_counter(&a.cnt->h_done, want);
}

// Failure-path check: the wait on a counter that nothing raises, with a short
// limit (about 1 ms).
__device__ unsigned int g_idle_counter;
__global__ void counter_timeout_probe_kernel(long long limit) { wait_counter(&g_idle_counter, 1u, limit); }

// What an epilogue warp needs for a CTA's run of blocks.
struct MoeBlocks {
  uint32_t tmem;         // two accumulator buffers of 128 columns
  uint64_t* tfull;
  uint32_t tempty;       // shared address
  float* sums;
  int n;                 // blocks
  int k0, act;           // the first one: block of its row of scales, (down) active expert
  int nt;                // (down) tile of 128 rows
  const float *pa, *pb;  // (up) scales of the tokens' codes and of the weights' row of blocks
};

// acc += scale * block sum over the run, for one token (lane) and 64 columns
// per thread; then the sums go to shared memory.  Scales come in groups of at
// most four blocks of one row, requested a group ahead (16-byte loads where
// the rows are aligned).  Down: the scale of h times that of the weights times
// the routing weight; a token that did not choose the block's expert has the
// weight -1, h has no row for it, and its lane adds nothing.
template <bool UP, int ROW>
__device__ __forceinline__ void moe_block_sums(const MoeArgs& a, const MoeBlocks& q, int warp, int lane) {
  const int quad = warp & 3, half = warp >> 2;
  const int row = quad * 32 + lane;
  const bool busy = quad * 32 < a.T;
  const int t = min(row, a.T - 1);
  const uint32_t taddr = q.tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 64;
  const int len = UP ? a.HB : a.IB;
  const bool vec = (UP ? a.vec13 : a.vec2) != 0;
  const float* pa = UP ? q.pa + t * a.HB : nullptr;
  const float* pb = q.pb;
  int act = q.act, kb = q.k0, left = q.n;  // of the next group to request
  float w_next = 1.0f;
  // the arrays behind pa and pb, and their extents
  const float* ba = UP ? a.sx : a.sh;
  const float* bb = UP ? a.s13 : a.s2;
  const unsigned long long na =
      UP ? static_cast<unsigned long long>(a.T) * a.HB : static_cast<unsigned long long>(a.A) * a.T * a.IB;
  const unsigned long long nb = static_cast<unsigned long long>(UP ? 2 * a.E : a.E) * a.IB * a.HB;
  auto enter = [&]() {
    w_next = ld_in<float>(a.wt + act * a.T + t, a.wt, static_cast<unsigned>(a.A * a.T));
    pa = a.sh + (static_cast<size_t>(act) * a.T + t) * a.IB;
    pb = a.s2 + (static_cast<size_t>(moe_expert(a, act)) * a.HB + q.nt) * a.IB;
  };
  const auto a1 = [&](int k) { return ld_in<float>(pa + k, ba, na); };
  const auto b1 = [&](int k) { return ld_in<float>(pb + k, bb, nb); };
  if (!UP) enter();
  Fp8Scales sc;
  float w = 1.0f, w_req = 1.0f;    // of the current group, of the requested one
  int have = 0, skip_req = 0, have_req = 0;
  auto request = [&]() {
    have_req = 0;
    if (left <= 0) return;
    if (!UP && kb == len) {
      kb = 0;
      ++act;
      enter();
    }
    w_req = w_next;
    skip_req = vec ? kb & 3 : 0;
    have_req = min(min(4 - skip_req, len - kb), left);
    if (!UP && w_next < 0.0f) {
      sc.x = sc.w = make_float4(0.f, 0.f, 0.f, 0.f);
    } else if (vec) {
      sc.load4(pa + (kb & ~3), ba, na, pb + (kb & ~3), bb, nb);
    } else {
      const int k1 = min(kb + 1, len - 1), k2 = min(kb + 2, len - 1), k3 = min(kb + 3, len - 1);
      sc.x = make_float4(a1(kb), a1(k1), a1(k2), a1(k3));
      sc.w = make_float4(b1(kb), b1(k1), b1(k2), b1(k3));
    }
    kb += have_req;
    left -= have_req;
  };
  float acc[64];
#pragma unroll
  for (int j = 0; j < 64; ++j) acc[j] = 0.0f;
  bool ok = true;  // after a wait gave up: go through the motions without waiting
  request();
#pragma unroll 1
  for (int i = 0; i < q.n; ++i) {
    const int b = i & 1;
    if (have == 0) {
      sc.take();
      for (int j = 0; j < skip_req; ++j) sc.shift();
      have = have_req;
      w = w_req;
      request();
    }
    const bool on = UP || !(w < 0.0f);
    const float f = UP ? sc.f0 : sc.f0 * w;
    sc.shift();
    --have;
    // (lanes whose token chose the expert have loaded scales, others have not;
    // the tensor-memory loads are of whole warps)
    if (!UP) __syncwarp();
    if (ok)
      ok = mbar_wait_warp(&q.tfull[b], (i >> 1) & 1);
    else
      __syncwarp();
    tc_fence_after();
    if (busy) {
      uint32_t v[2][16];
      tmem_ld16(taddr + b * 128, v[0]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tmem_wait_ld16(v[c & 1]);
        if (c < 3) tmem_ld16(taddr + b * 128 + 16 * (c + 1), v[(c + 1) & 1]);
        if (c == 3) {
          tc_fence_before();
          mbar_arrive_lane0(q.tempty + 8 * b, lane);
        }
        if (on) {
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            fma2(acc[16 * c + j], acc[16 * c + j + 1], f, v[c & 1][j], v[c & 1][j + 1]);
        }
        if (!UP) __syncwarp();
      }
    } else {
      tc_fence_before();
      mbar_arrive_lane0(q.tempty + 8 * b, lane);
    }
  }
  // every MMA of this CTA has read its operands, so the ring takes the sums
  if (ok && row < a.T) {
    float* dst = q.sums + row * ROW + half * 64;
#pragma unroll
    for (int c = 0; c < 16; ++c)
      *reinterpret_cast<float4*>(dst + 4 * c) =
          make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kMinBlocks)
    moe_expert_kernel(const __grid_constant__ CUtensorMap xmap,     // xq    {H, T, 1}
                      const __grid_constant__ CUtensorMap w13map,   // w13   {H, I, 2 E}, 64 rows
                      const __grid_constant__ CUtensorMap hmap,     // hq    {I, T, A}
                      const __grid_constant__ CUtensorMap w2map,    // w2    {I, H, E}
                      const MoeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem;                            // STAGES x kXStage
  uint8_t* ws = xs + C::STAGES * C::kXStage;     // STAGES x kWStage
  float* sums = reinterpret_cast<float*>(smem);  // [tokens][kRow], once the ring is idle
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);  // landed (tx)
  uint64_t* empty = full + C::STAGES;            // MMAs done reading (commit)
  uint64_t* tfull = empty + C::STAGES;           // block sum ready (commit)   [2]
  uint64_t* tempty = tfull + 2;                  // block sum read (epilogue)  [2]
  uint64_t* done = tempty + 2;                   // every MMA complete (commit)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* ticket_slot = tmem_holder + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], C::kEpiWarps);
    }
    mbar_init(done, 1);
    fence_barrier_init();
    grid_dep_launch();
  }
  if (warp == C::kMma) {
    tmem_alloc(tmem_holder, 256);
    tmem_relinquish();
  }
  __syncwarp();
  cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
  grid_dep_wait();  // the routing, and the call before it
  if (threadIdx.x == 0 && rank == 0) {
    const unsigned t = atomicAdd(&a.cnt->ticket, 1u);
    for (int r = 0; r < kMoeCluster; ++r) st_cluster_u32(mapa_shared(smem_u32(ticket_slot), r), t);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int ticket = static_cast<int>(*ticket_slot);

  // this CTA's work
  const int n_active = min(__ldcg(a.active), a.A);
  const int group = 2 * a.ksplit;                    // CTAs of one 128-channel block of h
  const int per = kMoeCluster / group;               // such blocks per cluster
  const int per_expert = (a.IB + per - 1) / per;     // clusters per expert
  const int up_clusters = n_active * per_expert;
  const int down_tiles = a.HB;
  const bool up = ticket < up_clusters;
  int n = 0;                                         // blocks of K
  int expert = 0, slot = 0, ib = 0, half64 = 0, k0 = 0, nt = 0;
  if (up) {
    slot = ticket / per_expert;
    expert = moe_expert(a, slot);
    ib = (ticket - slot * per_expert) * per + rank / group;
    half64 = rank % group / a.ksplit;
    const int s = rank % a.ksplit;
    k0 = a.HB * s / a.ksplit;
    n = ib < a.IB ? a.HB * (s + 1) / a.ksplit - k0 : 0;
  } else if (ticket - up_clusters < down_tiles) {
    nt = ticket - up_clusters;
    const long long units = static_cast<long long>(n_active) * a.IB;
    k0 = static_cast<int>(units * rank / kMoeCluster);
    n = static_cast<int>(units * (rank + 1) / kMoeCluster) - k0;
  }
  const bool down = !up && ticket - up_clusters < down_tiles;
  const unsigned h_want = static_cast<unsigned>(up_clusters) * kMoeCluster;
  const bool epi = (warp & 3) < C::QUADS && warp < 8;

  if (warp == C::kProducer) {
    if (lane == 0 && n > 0) {
      const uint64_t pol_w = policy_evict_first();  // read once
      const uint64_t pol_x = policy_evict_last();
      const uint32_t bytes = C::kWStage + static_cast<uint32_t>(a.T) * 128u;
      auto load_w = [&](int i) {
        const int s = i % C::STAGES;
        mbar_arrive_expect_tx(&full[s], bytes);
        if (up) {
          const int row = ib * kFp8Block + half64 * 64;
          tma_load_3d(ws + s * C::kWStage, &w13map, (k0 + i) * 128, row, 2 * expert, &full[s], pol_w);
          tma_load_3d(ws + s * C::kWStage + 64 * 128, &w13map, (k0 + i) * 128, row, 2 * expert + 1,
                      &full[s], pol_w);
        } else {
          const int act = (k0 + i) / a.IB;
          tma_load_3d(ws + s * C::kWStage, &w2map, (k0 + i - act * a.IB) * 128, nt * 128,
                      moe_expert(a, act), &full[s], pol_w);
        }
      };
      auto load_x = [&](int i) {
        const int s = i % C::STAGES;
        if (up) {
          tma_load_3d(xs + s * C::kXStage, &xmap, (k0 + i) * 128, 0, 0, &full[s], pol_x);
        } else {
          const int act = (k0 + i) / a.IB;
          tma_load_3d(xs + s * C::kXStage, &hmap, (k0 + i - act * a.IB) * 128, 0, act, &full[s], pol_x);
        }
      };
      const int early = min(n, C::STAGES);
      for (int i = 0; i < early; ++i) load_w(i);  // the weights do not wait for h
      bool ok = up || moe_wait_h(a, h_want);
      if (!up) fence_proxy_async_all();           // h was written by ordinary stores
      int i = 0;
      for (; i < n && (ok || i < early); ++i) {
        if (i >= C::STAGES) {
          if (!mbar_wait(&empty[i % C::STAGES], ((i / C::STAGES) - 1) & 1)) break;
          load_w(i);
        }
        load_x(i);  // also after a wait gave up: the armed barriers must complete
      }
      // never leave with copies in flight
      for (int j = i - 1; j >= 0 && j >= i - C::STAGES; --j)
        mbar_wait(&full[j % C::STAGES], (j / C::STAGES) & 1);
    }
  } else if (warp == C::kMma) {
    constexpr uint32_t idesc = idesc_e4m3_f32(128, 128);
    const uint64_t xd0 = smem_desc_sw128(smem_u32(xs)), wd0 = smem_desc_sw128(smem_u32(ws));
    int s = 0;
    uint32_t phase = 0;
    for (int i = 0; i < n; ++i) {
      const int b = i & 1;
      if (!mbar_wait_warp(&full[s], phase) ||
          (i >= 2 && !mbar_wait_warp(&tempty[b], ((i >> 1) - 1) & 1)))
        break;
      tc_fence_after();
      const uint64_t xd = xd0 + static_cast<uint32_t>(s) * (C::kXStage >> 4);
      const uint64_t wd = wd0 + static_cast<uint32_t>(s) * (C::kWStage >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8_ss(tmem + b * 128, xd + 2 * kk, wd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
        mma_commit(&empty[s]);
        mma_commit(&tfull[b]);
      }
      __syncwarp();
      if (++s == C::STAGES) {
        s = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) mma_commit(done);
    __syncwarp();
  } else if (epi && n > 0) {
    MoeBlocks q{};
    q.tmem = tmem;
    q.tfull = tfull;
    q.tempty = smem_u32(&tempty[0]);
    q.sums = sums;
    q.n = n;
    if (up) {
      const int half = warp >> 2;
      q.k0 = k0;
      q.pa = a.sx;
      q.pb = a.s13 + (static_cast<size_t>(2 * expert + half) * a.IB + ib) * a.HB;
      moe_block_sums<true, C::kRow>(a, q, warp, lane);
    } else if (__all_sync(0xffffffffu, lane != 0 || moe_wait_h(a, h_want))) {
      __syncwarp();  // (a vote alone orders no memory: lane 0 has seen h published)
      q.act = k0 / a.IB;
      q.k0 = k0 - q.act * a.IB;
      q.nt = nt;
      moe_block_sums<false, C::kRow>(a, q, warp, lane);
    } else {
      // h never came: let the MMA warp go on without reading its sums
      for (int i = 0; i < n; ++i) {
        if (!mbar_wait_warp(&tfull[i & 1], (i >> 1) & 1)) break;
        mbar_arrive_lane0(smem_u32(&tempty[0]) + 8 * (i & 1), lane);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // the cluster's sums are in place

  if (up) {
    // a warp per token: 4 of the block's 128 channels per lane, gate and up
    // summed over the K ranges in order, h, its largest, its codes
    const int g0 = rank - rank % group;  // first CTA of this block's group
    const uint32_t mine = smem_u32(sums);
    if (ib < a.IB) {
      for (int t = (rank - g0) * C::kWarps + warp; t < a.T; t += group * C::kWarps) {
        if (ld_in<float>(a.wt + slot * a.T + t, a.wt, static_cast<unsigned>(a.A * a.T)) < 0.0f) continue;
        const int owner = g0 + (lane >> 4) * a.ksplit;
        const uint32_t at = mine + static_cast<uint32_t>(t * C::kRow + (lane & 15) * 4) * 4u;
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
        for (int s = 0; s < a.ksplit; ++s) {
          const float4 gv = ld_cluster_f4(mapa_shared(at, owner + s));
          const float4 uv = ld_cluster_f4(mapa_shared(at + 256, owner + s));
          g.x += gv.x; g.y += gv.y; g.z += gv.z; g.w += gv.w;
          u.x += uv.x; u.y += uv.y; u.z += uv.z; u.w += uv.w;
        }
        const float gg[4] = {g.x, g.y, g.z, g.w}, uu[4] = {u.x, u.y, u.z, u.w};
        float h[4];
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = __fdiv_rn(gg[j], 1.0f + expf(-gg[j])) * uu[j];
          mx = max(mx, abs_bits(h[j]));
        }
        mx = __reduce_max_sync(0xffffffffu, mx);
        const float sc = fp8_scale(mx);
        const size_t hrow = static_cast<size_t>(slot) * a.T + t;
        const int c = ib * kFp8Block + lane * 4;
        const unsigned long long rows = static_cast<unsigned long long>(a.A) * a.T;
        if (c < a.I)
          st_in(a.hq + hrow * a.I + c, a.hq, rows * a.I,
                e4m3x2(__fdiv_rn(h[0], sc), __fdiv_rn(h[1], sc)) |
                    (e4m3x2(__fdiv_rn(h[2], sc), __fdiv_rn(h[3], sc)) << 16));
        if (lane == 0) st_in(a.sh + hrow * a.IB + ib, a.sh, rows * a.IB, sc);
      }
    }
    // publish: ordinary stores, read elsewhere by tensor copies and loads
    fence_proxy_async_all();
    __syncthreads();
    if (threadIdx.x == 0) red_add_release_gpu(&a.cnt->h_done, 1u);
  } else if (down) {
    const int q0 = 32 * rank / kMoeCluster, w = 32 / kMoeCluster;  // in units of 4 columns
    const uint32_t mine = smem_u32(sums);
    const long long units = static_cast<long long>(n_active) * a.IB;
    for (int e = threadIdx.x; e < a.T * w; e += C::kThreads) {
      const int r = e / w, c = (q0 + e - r * w) * 4;
      const uint32_t at = mine + static_cast<uint32_t>(r * C::kRow + c) * 4u;
      float4 v[kMoeCluster];
#pragma unroll
      for (int p = 0; p < kMoeCluster; ++p)  // (an empty K range left no sums)
        v[p] = units * p / kMoeCluster < units * (p + 1) / kMoeCluster
                   ? ld_cluster_f4(mapa_shared(at, p))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < kMoeCluster; ++p) {
        sum.x += v[p].x;
        sum.y += v[p].y;
        sum.z += v[p].z;
        sum.w += v[p].w;
      }
      const int col = nt * 128 + c;
      uint16_t* y = a.Y + static_cast<size_t>(r) * a.H + col;
      const unsigned long long n_y = static_cast<unsigned long long>(a.T) * a.H;
      if (a.vec && col + 4 <= a.H) {
        st_in(y, a.Y, n_y, make_uint2(bf16_pack2(sum.x, sum.y), bf16_pack2(sum.z, sum.w)));
      } else {
        const float s4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < a.H) st_in(y + j, a.Y, n_y, __bfloat16_as_ushort(__float2bfloat16_rn(s4[j])));
      }
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another reads its sums
  if (threadIdx.x == 0 && rank == 0) {
    const unsigned clusters = gridDim.x / kMoeCluster;
    if (atom_add_acq_rel_gpu(&a.cnt->left, 1u) == clusters - 1) {
      // the last cluster leaves the counters as it found them
      a.cnt->ticket = 0u;
      a.cnt->h_done = 0u;
      a.cnt->left = 0u;
    }
  }
  if (warp == C::kMma) {
    mbar_wait_warp(done, 0);  // every issued MMA has completed
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace w4
