// w4_fp8_gemm.cuh -- Y[m,n] = sum over 128-channel blocks j of
//   sx[m,j] * sw[n/128,j] * sum over k in j of qx[m,k] * qw[n,k]
// for e4m3 codes, on the tensor cores (tcgen05.mma kind::f8f6f4).
//
// The scales change every 128 channels, so the tensor-memory accumulator
// holds one block's sum at a time: four MMAs of K = 32 fill one of two
// accumulator buffers while the epilogue warps read the other and add
//   acc += (sx sw) * block sum
// to fp32 registers, one fma per output and block.  Tokens are the MMA's rows
// (tensor-memory lanes) and weight rows its columns: a thread then owns one
// token, sx is one register, sw one value per warp and block (its columns lie
// in one block of 128 weight rows), and few tokens cost nothing but idle
// lanes, which a call bound by its weight stream has to spare.
//
// Tiles of 128 tokens x NT weight rows per CTA, or, for more than 128 tokens,
// CTA pairs (cta_group::2) of 256 x 256 with each CTA staging half of each
// operand.  A stage is one block of 128 channels: both operands arrive by TMA
// as rows of 128 bytes in the 128-byte swizzle (channels and rows past the
// end read as zero).  Warp 0 issues the copies, warp 1 the MMAs, 8 warps are
// the epilogue (4 tensor-memory lane quadrants x 2 column halves).
//
// Work: a persistent grid.  Each worker (CTA or pair) takes whole tiles while
// every worker gets one; the tiles left over are cut along K into equal runs
// of blocks, one per worker, whose fp32 partial sums the last run of a tile
// to finish adds in the order of K (the result does not depend on which
// that is).
#pragma once

#include <cuda_bf16.h>

#include "w4_fp8.cuh"

namespace w4 {

constexpr int kFp8Rows = 128;        // tokens per CTA tile (tensor-memory lanes)
constexpr int kFp8EpiWarps = 8;
constexpr uint16_t kFp8PairMask = 0x3;

template <int NT_, bool PAIR_, int STAGES_>
struct Fp8Cfg {
  static constexpr int NT = NT_;            // weight rows (MMA columns) per tile
  static constexpr bool PAIR = PAIR_;
  static constexpr int STAGES = STAGES_;
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kWRows = NT / kCtas;  // weight rows this CTA stages
  static constexpr int kXStage = kFp8Rows * 128;
  static constexpr int kWStage = kWRows * 128;
  static constexpr int kThreads = 64 + kFp8EpiWarps * 32;
  static constexpr int kCols = NT / 2;       // columns per epilogue thread
  static constexpr int kTmemCols = 2 * NT;
  static constexpr int kSmemBytes = 1024 + STAGES * (kXStage + kWStage) + (2 * STAGES + 5) * 8 + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Fp8GemmArgs {
  const float* sx;        // [M, KB]
  const float* sw;        // [NB, KB]
  uint16_t* Y;            // bf16 [M, N]
  float* partial;         // [slot][rows][NT]: two slots per worker (and CTA of a pair)
  unsigned int* counter;  // [tail tile (and CTA of a pair)], zero between calls
  int M, N, KB, NB;
  int tiles_m, tiles_n, group_m;
  int workers;            // CTAs or pairs
  int rounds;             // whole tiles per worker
  int tail;               // tiles left over, the last ones
  int tail_workers;       // runs they are cut into (0: each whole, one worker each)
  int rows;               // rows of a partial slot
  int vec;                // Y rows take 16-byte stores
  int keep_w;             // weights are read by several token tiles: keep them in L2
  unsigned long long partial_floats;  // extent, for the bounds-checked build
};

// One piece of a worker's work: blocks [k0, k1) of a tile.
struct Fp8Piece {
  int tile, k0, k1;
};

// The pieces of a worker in order: whole tiles, then its run of the tail.
struct Fp8Work {
  const Fp8GemmArgs& a;
  int w, round;
  long long u, end;
  __device__ __forceinline__ Fp8Work(const Fp8GemmArgs& args, int worker)
      : a(args), w(worker), round(0), u(0), end(0) {
    if (a.tail_workers > 0 && w < a.tail_workers) {
      u = run_start(w);
      end = run_start(w + 1);
    }
  }
  __device__ __forceinline__ long long units() const { return static_cast<long long>(a.tail) * a.KB; }
  __device__ __forceinline__ long long run_start(int c) const { return units() * c / a.tail_workers; }
  // the worker whose run holds unit v
  __device__ __forceinline__ int run_of(long long v) const {
    return static_cast<int>(((v + 1) * a.tail_workers - 1) / units());
  }
  __device__ __forceinline__ bool next(Fp8Piece& p) {
    const int whole = a.rounds + (a.tail_workers == 0 && w < a.tail ? 1 : 0);
    if (round < whole) {
      p.tile = w + round * a.workers;
      p.k0 = 0;
      p.k1 = a.KB;
      ++round;
      return true;
    }
    if (u >= end) return false;
    const int t = static_cast<int>(u / a.KB);
    p.tile = a.rounds * a.workers + t;
    p.k0 = static_cast<int>(u - static_cast<long long>(t) * a.KB);
    const long long left = end - u;
    p.k1 = left < a.KB - p.k0 ? p.k0 + static_cast<int>(left) : a.KB;
    u += p.k1 - p.k0;
    return true;
  }
  // token and weight tile of a tile index: groups of group_m token tiles, the
  // token tile fastest, so that the tiles running together share their weight
  // tiles and few token tiles through L2
  __device__ __forceinline__ void tile_at(int t, int& mt, int& nt) const {
    const int gsize = a.group_m * a.tiles_n;
    const int g = t / gsize;
    const int gm = min(a.group_m, a.tiles_m - g * a.group_m);
    const int lin = t - g * gsize;
    nt = lin / gm;
    mt = g * a.group_m + lin - nt * gm;
  }
};

__device__ __forceinline__ void epi_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

__device__ __forceinline__ uint32_t bf16_pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    fp8_tc_gemm_kernel(const __grid_constant__ CUtensorMap xmap,
                       const __grid_constant__ CUtensorMap wmap, const Fp8GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem;                                   // STAGES x kXStage
  uint8_t* ws = xs + C::STAGES * C::kXStage;            // STAGES x kWStage
  uint64_t* full = reinterpret_cast<uint64_t*>(ws + C::STAGES * C::kWStage);  // landed (tx)
  uint64_t* empty = full + C::STAGES;                   // MMAs done reading (commit)
  uint64_t* tfull = empty + C::STAGES;                  // block sum ready (commit)  [2]
  uint64_t* tempty = tfull + 2;                         // block sum read (8 or 16 warps) [2]
  uint64_t* done = tempty + 2;                          // every MMA complete (commit)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  int* last_flag = reinterpret_cast<int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = C::PAIR ? cluster_ctarank() : 0u;
  const int worker = static_cast<int>(blockIdx.x) / C::kCtas;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], C::kCtas * kFp8EpiWarps);
    }
    mbar_init(done, 1);
    fence_barrier_init();
    grid_dep_launch();
  }
  if (warp == 1) {
    if constexpr (C::PAIR) {
      tmem_alloc_pair(tmem_holder, C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, C::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (C::PAIR)
    cluster_sync();  // the peer's copies and arrivals target this CTA's barriers
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  Fp8Work work(a, worker);
  Fp8Piece p;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&wmap);
      prefetch_tensormap(&xmap);
      const uint64_t pol_w = a.keep_w ? policy_evict_normal() : policy_evict_first();
      const uint64_t pol_x = policy_evict_last();
      constexpr uint32_t kBytes = C::kCtas * C::kWStage;
      // the X box may be shorter than the stage's 128 rows; its bytes are counted as copied
      const uint32_t x_bytes = static_cast<uint32_t>(C::kCtas) * static_cast<uint32_t>(a.rows) * 128u;
      auto arm = [&](int s) {  // a pair: the leader's barrier counts both CTAs' bytes
        if (rank == 0) mbar_arrive_expect_tx(&full[s], kBytes + x_bytes);
      };
      auto load_w = [&](int s, int nt, int kb) {
        if constexpr (C::PAIR)
          tma_load_3d_pair(ws + s * C::kWStage, &wmap, kb * 128,
                           nt * C::NT + static_cast<int>(rank) * C::kWRows, 0,
                           mapa_shared(smem_u32(&full[s]), 0), pol_w);
        else
          tma_load_3d(ws + s * C::kWStage, &wmap, kb * 128, nt * C::NT, 0, &full[s], pol_w);
      };
      auto load_x = [&](int s, int mt, int kb) {
        const int m = (mt * C::kCtas + static_cast<int>(rank)) * kFp8Rows;
        if constexpr (C::PAIR)
          tma_load_3d_pair(xs + s * C::kXStage, &xmap, kb * 128, m, 0,
                           mapa_shared(smem_u32(&full[s]), 0), pol_x);
        else
          tma_load_3d(xs + s * C::kXStage, &xmap, kb * 128, m, 0, &full[s], pol_x);
      };
      // the weights do not depend on the previous kernel: the first ring of
      // them is requested before the dependency wait
      int early = 0;
      {
        Fp8Work w2 = work;
        while (early < C::STAGES && w2.next(p)) {
          int mt, nt;
          w2.tile_at(p.tile, mt, nt);
          for (int kb = p.k0; kb < p.k1 && early < C::STAGES; ++kb, ++early) {
            arm(early);
            load_w(early, nt, kb);
          }
        }
      }
      grid_dep_wait();
      int it = 0;
      bool ok = true;
      while (ok && work.next(p)) {
        int mt, nt;
        work.tile_at(p.tile, mt, nt);
        for (int kb = p.k0; kb < p.k1; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (it >= C::STAGES) {
            if (!mbar_wait(&empty[s], ((it / C::STAGES) - 1) & 1)) {
              ok = false;
              break;
            }
            arm(s);
            load_w(s, nt, kb);
          }
          load_x(s, mt, kb);
        }
      }
      // never leave with copies in flight (a pair: the leader's barriers count
      // both CTAs'), nor before the last arrivals on this CTA's own barriers
      if (rank == 0)
        for (int i = it - 1; i >= 0 && i >= it - C::STAGES; --i)
          mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1);
      for (int i = it - 1; i >= 0 && i >= it - C::STAGES; --i)
        if (!mbar_wait(&empty[i % C::STAGES], (i / C::STAGES) & 1)) break;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(C::kCtas * 128, C::NT);
      int it = 0;
      bool ok = true;
      while (ok && work.next(p)) {
        for (int kb = p.k0; kb < p.k1; ++kb, ++it) {
          const int s = it % C::STAGES, b = it & 1;
          if (!mbar_wait(&full[s], (it / C::STAGES) & 1) ||
              (it >= 2 && !mbar_wait(&tempty[b], ((it >> 1) - 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t xa = smem_u32(xs + s * C::kXStage);
          const uint32_t wa = smem_u32(ws + s * C::kWStage);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (C::PAIR)
              mma_f8_ss_pair(tmem + b * C::NT, smem_desc_sw128(xa + kk * 32),
                             smem_desc_sw128(wa + kk * 32), idesc, kk > 0 ? 1u : 0u);
            else
              mma_f8_ss(tmem + b * C::NT, smem_desc_sw128(xa + kk * 32),
                        smem_desc_sw128(wa + kk * 32), idesc, kk > 0 ? 1u : 0u);
          }
          if constexpr (C::PAIR) {
            mma_commit_pair(&empty[s], kFp8PairMask);
            mma_commit_pair(&tfull[b], kFp8PairMask);
          } else {
            mma_commit(&empty[s]);
            mma_commit(&tfull[b]);
          }
        }
      }
      if constexpr (C::PAIR)
        mma_commit_pair(done, kFp8PairMask);
      else
        mma_commit(done);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;                 // tensor-memory lanes 32 quad ..
    const int half = (warp - 2) >> 2;          // columns half * NT/2 ..
    const int row = quad * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * C::kCols;
    bool ok = true;  // after a wait gave up: go through the motions without waiting
    int it = 0;
    grid_dep_wait();
    while (work.next(p)) {
      int mt, nt;
      work.tile_at(p.tile, mt, nt);
      const int m0 = (mt * C::kCtas + static_cast<int>(rank)) * kFp8Rows;
      const int rows = min(kFp8Rows, a.M - m0);  // may be <= 0 in a pair's second CTA
      const bool busy = quad * 32 < rows;
      const int m = m0 + row, n0 = nt * C::NT + half * C::kCols;
      const float* sxp = a.sx + static_cast<size_t>(min(m, a.M - 1)) * a.KB;
      const float* swp = a.sw + static_cast<size_t>(min(n0 / kFp8Block, a.NB - 1)) * a.KB;
      float acc[C::kCols];
#pragma unroll
      for (int j = 0; j < C::kCols; ++j) acc[j] = 0.0f;
      float sx_next = __ldg(sxp + p.k0), sw_next = __ldg(swp + p.k0);
      for (int kb = p.k0; kb < p.k1; ++kb, ++it) {
        const int b = it & 1;
        const float f = sx_next * sw_next;
        const int kn = min(kb + 1, p.k1 - 1);
        sx_next = __ldg(sxp + kn);
        sw_next = __ldg(swp + kn);
        if (ok && !__all_sync(0xffffffffu, mbar_wait(&tfull[b], (it >> 1) & 1))) ok = false;
        tc_fence_after();
        if (busy) {
          uint32_t v[2][16];
          tmem_ld16(taddr + b * C::NT, v[0]);
#pragma unroll
          for (int c = 0; c < C::kCols / 16; ++c) {
            tmem_wait_ld16(v[c & 1]);
            if (c + 1 < C::kCols / 16) tmem_ld16(taddr + b * C::NT + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              acc[16 * c + j] = fmaf(f, __uint_as_float(v[c & 1][j]), acc[16 * c + j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (C::PAIR)
            mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[b]), 0));  // the leader's
          else
            mbar_arrive(&tempty[b]);
        }
      }
      if (p.k0 == 0 && p.k1 == a.KB) {
        if (row < rows) {
          uint16_t* y = a.Y + static_cast<size_t>(m) * a.N + n0;
#pragma unroll
          for (int c = 0; c < C::kCols / 8; ++c) {
            const int n = n0 + 8 * c;
            if (a.vec && n + 8 <= a.N) {
              uint4 o;
              o.x = bf16_pack2(acc[8 * c], acc[8 * c + 1]);
              o.y = bf16_pack2(acc[8 * c + 2], acc[8 * c + 3]);
              o.z = bf16_pack2(acc[8 * c + 4], acc[8 * c + 5]);
              o.w = bf16_pack2(acc[8 * c + 6], acc[8 * c + 7]);
              *reinterpret_cast<uint4*>(y + 8 * c) = o;
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (n + j < a.N)
                  y[8 * c + j] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[8 * c + j]));
            }
          }
        }
        continue;
      }
      // a run of the tail: publish the partial sums; the last run of the tile
      // to arrive adds them in the order of K
      const int tt = p.tile - a.rounds * a.workers;
      const long long ubase = static_cast<long long>(tt) * a.KB;
      const int first = work.run_of(ubase), last = work.run_of(ubase + a.KB - 1);
      // a worker's run starts in this tile, or ends here after the one before
      auto slot_of = [&](int c) -> size_t {
        const size_t idx = work.run_start(c) < ubase ? 1 : 0;
        return ((static_cast<size_t>(c) * 2 + idx) * C::kCtas + rank) * static_cast<size_t>(a.rows) * C::NT;
      };
      const size_t mine = slot_of(worker);
      if (row < rows) {
        float* dst = a.partial + mine + static_cast<size_t>(row) * C::NT + half * C::kCols;
        if (in_bounds(mine + static_cast<size_t>(row) * C::NT + C::NT - 1, a.partial_floats)) {
#pragma unroll
          for (int c = 0; c < C::kCols / 4; ++c)
            *reinterpret_cast<float4*>(dst + 4 * c) =
                make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
        }
      }
      __threadfence();
      epi_sync();
      if (threadIdx.x == 64) {
        unsigned int* ctr = a.counter + tt * C::kCtas + static_cast<int>(rank);
        const unsigned prev = atom_add_acq_rel_gpu(ctr, 1u);
        const bool is_last = prev == static_cast<unsigned>(last - first);
        if (is_last) *ctr = 0u;  // leave the workspace zeroed
        *last_flag = is_last ? 1 : 0;
      }
      epi_sync();
      if (*last_flag) {
        __threadfence();
        constexpr int kQ = C::NT / 4;
        const size_t s0 = slot_of(first);
        const size_t cstep = 2 * static_cast<size_t>(C::kCtas) * a.rows * C::NT;
        // runs after the first start inside this tile: their first slots
        const size_t s1 = ((static_cast<size_t>(first) * 2) * C::kCtas + rank) *
                          static_cast<size_t>(a.rows) * C::NT;
        for (int e = static_cast<int>(threadIdx.x) - 64; e < rows * kQ; e += kFp8EpiWarps * 32) {
          const int r = e / kQ, c4 = (e - r * kQ) * 4;
          const size_t at = static_cast<size_t>(r) * C::NT + c4;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = first; c <= last; ++c) {
            const size_t src = (c == first ? s0 : s1 + (c - first) * cstep) + at;
            if (!in_bounds(src + 3, a.partial_floats)) continue;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(a.partial + src));
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
          }
          const int n = nt * C::NT + c4;
          uint16_t* y = a.Y + static_cast<size_t>(m0 + r) * a.N + n;
          if (a.vec && n + 4 <= a.N) {
            *reinterpret_cast<uint2*>(y) = make_uint2(bf16_pack2(sum.x, sum.y), bf16_pack2(sum.z, sum.w));
          } else {
            const float s4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n + j < a.N) y[j] = __bfloat16_as_ushort(__float2bfloat16_rn(s4[j]));
          }
        }
      }
    }
  }

  tc_fence_before();
  if constexpr (C::PAIR)
    cluster_sync();  // neither CTA leaves while the other may reach its memory
  else
    __syncthreads();
  if (warp == 1) {
    mbar_wait(done, 0);  // every issued MMA has completed
    tc_fence_after();
    if constexpr (C::PAIR)
      tmem_dealloc_pair(tmem, C::kTmemCols);
    else
      tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace w4
