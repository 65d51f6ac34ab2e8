// w4_fp8_gemm.cuh -- Y[m,n] = sum over 128-channel blocks j of
//   sx[m,j] * sw[n/128,j] * sum over k in j of qx[m,k] * qw[n,k]
// for e4m3 codes, on the tensor cores (tcgen05.mma kind::f8f6f4).
//
// The scales change every 128 channels, so the tensor-memory accumulator
// holds one block's sum at a time: four MMAs of K = 32 fill one
// accumulator buffer while the epilogue warps read another and add
//   acc += (sx sw) * block sum
// to fp32 registers, one fma per output and block.  Tokens are the MMA's rows
// (tensor-memory lanes) and weight rows its columns: a thread then owns one
// token, sx is one register, sw one value per warp and block (its columns lie
// in one block of 128 weight rows), and few tokens cost nothing but idle
// lanes, which a call bound by its weight stream has to spare.
//
// A stage is one block of 128 channels: both operands arrive by TMA as rows of
// 128 bytes in the 128-byte swizzle (channels and rows past the end read as
// zero).  One warp issues the copies, one the MMAs, the epilogue warps are the
// used tensor-memory lane quadrants x 2 column halves.
//
// Up to 128 tokens (fp8_rows_gemm_kernel): one tile of all tokens x 128 weight
// rows per cluster, whose CTAs take a K range each and add their sums over
// distributed shared memory.
//
// More tokens (fp8_tc_gemm_kernel): CTA pairs (cta_group::2) of 256 tokens x
// 256 or 128 weight rows, each CTA staging half of each operand, in a
// persistent grid.  Each pair takes whole tiles while every pair gets one; the
// tiles left over stay whole or are cut along K into equal runs of blocks, whose
// fp32 partial sums the last run of a tile to finish adds in the order of K (the
// result does not depend on which that is).
//
// Measured on B200, per call.  Up to 64 tokens about 5.5 us that do not depend on
// K, then the weights: 1 x 12288 x 4096 12.5 us, 4.0 TB/s; 33 x 4096 x 11008
// 14.5 us (5.3 TB/s for what K adds).  128 x 12288 x 4096 18.2 us: 96 tiles on
// 148 SMs, 0.41 us per block of a CTA.  2048 x 28672 x 8192 470 to 515 us (1.87
// to 2.05 PFLOP/s) in short runs, 550 us (1.75 PFLOP/s) in a loop of seconds,
// where the 1000 W limit takes the SMs to 1.57 GHz.  A pair's block takes 0.56 us:
// bound by the hand-over of the two accumulator buffers (0.50 us with no loads)
// and by the operands' way through L2 (0.456 us with no read-out).  With 256
// weight rows the epilogue warps' 128 running sums leave 44 bytes on the stack.
#pragma once

#include <cuda_bf16.h>

#include "w4_fp8.cuh"

namespace w4 {

constexpr int kFp8Rows = 128;        // tokens per CTA tile (tensor-memory lanes)
constexpr int kFp8EpiWarps = 8;
constexpr uint16_t kFp8PairMask = 0x3;

// A CTA pair's tile: 256 tokens x NT weight rows.  NT = 256 moves the fewest
// operand bytes through L2 per product; NT = 128 leaves smaller tiles, which
// fill the last wave of a few better.
template <int NT_, int STAGES_>
struct Fp8Cfg {
  static constexpr int NT = NT_;             // weight rows (MMA columns) per tile
  static constexpr int STAGES = STAGES_;
  static constexpr int kWRows = NT / 2;      // weight rows this CTA stages
  static constexpr int kXStage = kFp8Rows * 128;
  static constexpr int kWStage = kWRows * 128;
  static constexpr int kThreads = 128 + kFp8EpiWarps * 32;
  static constexpr int kCols = NT / 2;       // columns (running sums) per epilogue thread
  static constexpr int kBufs = 512 / NT;     // block sums in tensor memory, all 512 columns
  // 128 running sums per thread need registers from the first warpgroup:
  // (120 + 2 * 192) * 128 = 168 * 384 threads
  static constexpr bool kRegSplit = NT == 256;
  static constexpr int kLaunchRegs = 168, kFewRegs = 120, kManyRegs = 192;
  static_assert(kFewRegs * 128 + kManyRegs * 256 <= kLaunchRegs * kThreads, "register shares");
  // per epilogue warp, a box of 32 tokens x 64 outputs in bf16 (128-byte rows)
  // in the 128-byte swizzle
  static constexpr int kYWarp = 32 * 64 * 2;
  static constexpr int kSmemBytes = 1024 + STAGES * (kXStage + kWStage) + kFp8EpiWarps * kYWarp +
                                    (2 * STAGES + 2 * kBufs + 1) * 8 + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Fp8GemmArgs {
  const float* sx;        // [M, KB]
  const float* sw;        // [NB, KB]
  uint16_t* Y;            // bf16 [M, N]
  float* partial;         // two slots of 128 tokens x NT per worker and CTA of the pair
  unsigned int* counter;  // [tail tile (and CTA of a pair)], zero between calls
  int M, N, KB, NB;
  int tiles_m, tiles_n, group_m;
  int workers;            // pairs
  int rounds;             // whole tiles per worker
  int tail;               // tiles left over, the last ones
  int tail_workers;       // runs they are cut into (0: each whole, one worker each)
  int vec_s;              // sx and sw rows are 16-byte aligned
  int vec;                // Y rows are 16-byte aligned: tensor copies and vector stores
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
  int u, end;  // (the host cuts a tail only where units * workers fits in 31 bits)
  __device__ __forceinline__ Fp8Work(const Fp8GemmArgs& args, int worker)
      : a(args), w(worker), round(0), u(0), end(0) {
    if (a.tail_workers > 0 && w < a.tail_workers) {
      u = run_start(w);
      end = run_start(w + 1);
    }
  }
  __device__ __forceinline__ int units() const { return a.tail * a.KB; }
  __device__ __forceinline__ int run_start(int c) const { return units() * c / a.tail_workers; }
  // the worker whose run holds unit v
  __device__ __forceinline__ int run_of(int v) const {
    return ((v + 1) * a.tail_workers - 1) / units();
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
    const int t = u / a.KB;
    p.tile = a.rounds * a.workers + t;
    p.k0 = u - t * a.KB;
    p.k1 = min(a.KB, p.k0 + end - u);
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
  __syncwarp();  // (the barrier is of whole warps)
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
                       const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap ymap, const Fp8GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem;                                   // STAGES x kXStage
  uint8_t* ws = xs + C::STAGES * C::kXStage;            // STAGES x kWStage
  uint8_t* ys = ws + C::STAGES * C::kWStage;            // 8 x kYWarp
  uint64_t* full = reinterpret_cast<uint64_t*>(ys + kFp8EpiWarps * C::kYWarp);  // landed (tx)
  uint64_t* empty = full + C::STAGES;                   // MMAs done reading (commit)
  uint64_t* tfull = empty + C::STAGES;                  // block sum ready (commit)       [kBufs]
  uint64_t* tempty = tfull + C::kBufs;                  // block sum read (both CTAs' warps) [kBufs]
  uint64_t* done = tempty + C::kBufs;                   // every MMA complete (commit)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  int* last_flag = reinterpret_cast<int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int worker = static_cast<int>(blockIdx.x) / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kFp8EpiWarps);
    }
    mbar_init(done, 1);
    fence_barrier_init();
    grid_dep_launch();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // the peer's copies and arrivals target this CTA's barriers
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  Fp8Work work(a, worker);
  Fp8Piece p;

  if (C::kRegSplit && warp < 4) regs_dec<C::kFewRegs>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&wmap);
      prefetch_tensormap(&xmap);
      const uint64_t pol_w = a.keep_w ? policy_evict_normal() : policy_evict_first();
      const uint64_t pol_x = policy_evict_last();
      constexpr uint32_t kBytes = 2 * (C::kXStage + C::kWStage);
      auto arm = [&](int s) {  // a pair: the leader's barrier counts both CTAs' bytes
        if (rank == 0) mbar_arrive_expect_tx(&full[s], kBytes);
      };
      auto w_row = [&](int nt) { return nt * C::NT + static_cast<int>(rank) * C::kWRows; };
      auto load_w = [&](int s, int nt, int kb) {
        tma_load_3d_pair(ws + s * C::kWStage, &wmap, kb * 128, w_row(nt), 0,
                         mapa_shared(smem_u32(&full[s]), 0), pol_w);
      };
      auto load_x = [&](int s, int mt, int kb) {
        const int m = (mt * 2 + static_cast<int>(rank)) * kFp8Rows;
        tma_load_3d_pair(xs + s * C::kXStage, &xmap, kb * 128, m, 0,
                         mapa_shared(smem_u32(&full[s]), 0), pol_x);
      };
      // before the dependency wait the first ring of weights is on its way into
      // L2; they are read after it, like everything that a kernel ahead on the
      // stream may have written
      {
        Fp8Work w2 = work;
        int early = 0;
        while (early < C::STAGES && w2.next(p)) {
          int mt, nt;
          w2.tile_at(p.tile, mt, nt);
          for (int kb = p.k0; kb < p.k1 && early < C::STAGES; ++kb, ++early)
            tma_prefetch_3d(&wmap, kb * 128, w_row(nt), 0, pol_w);
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
          if (it >= C::STAGES && !mbar_wait(&empty[s], ((it / C::STAGES) - 1) & 1)) {
            ok = false;
            break;
          }
          arm(s);
          load_w(s, nt, kb);
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
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(2 * 128, C::NT);
      const uint64_t xd0 = smem_desc_sw128(smem_u32(xs)), wd0 = smem_desc_sw128(smem_u32(ws));
      int s = 0;
      uint32_t it = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && work.next(p)) {
        for (int kb = p.k0; kb < p.k1; ++kb, ++it) {
          const uint32_t b = it & (C::kBufs - 1);
          ok = mbar_wait_warp(&full[s], phase) &&
               (it < C::kBufs || mbar_wait_warp(&tempty[b], ((it / C::kBufs) - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          // descriptor addresses are in units of 16 bytes
          const uint64_t xd = xd0 + static_cast<uint32_t>(s) * (C::kXStage >> 4);
          const uint64_t wd = wd0 + static_cast<uint32_t>(s) * (C::kWStage >> 4);
          const uint32_t d = tmem + b * C::NT;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              mma_f8_ss_pair(d, xd + 2 * kk, wd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit_pair(&empty[s], kFp8PairMask);
            mma_commit_pair(&tfull[b], kFp8PairMask);
          }
          __syncwarp();
          if (++s == C::STAGES) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (elect_one()) {
        mma_commit_pair(done, kFp8PairMask);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    if (C::kRegSplit) regs_inc<C::kManyRegs>();
    const int quad = warp & 3;                 // tensor-memory lanes 32 quad ..
    const int half = (warp - 4) >> 2;          // columns half * NT/2 ..
    const int row = quad * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * C::kCols;
    uint8_t* yw = ys + (warp - 4) * C::kYWarp;
    bool ok = true;  // after a wait gave up: go through the motions without waiting
    uint32_t it = 0;
    // this warp has read accumulator buffer b
    // (a pair: on the leader's barrier)
    const uint32_t te0 = mapa_shared(smem_u32(&tempty[0]), 0);
    auto release = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      mbar_arrive_cluster_lane0(te0 + 8 * b, lane);
    };
    // Scales, four blocks at a time and four ahead: a token's are contiguous, so
    // the 32 lanes' loads touch 32 lines, and shared memory and L1 have one data
    // path that the operands already fill; 16-byte loads make that a quarter.
    const float *sxp = nullptr, *swp = nullptr;
    int mt = 0, nt = 0;
    float4 sx4, sw4;  // of the next group of four
    const auto x1 = [&](int g) {
      return ld_in<float>(sxp + g, a.sx, static_cast<unsigned long long>(a.M) * a.KB);
    };
    const auto w1 = [&](int g) {
      return ld_in<float>(swp + g, a.sw, static_cast<unsigned long long>(a.NB) * a.KB);
    };
    auto scales = [&](int g) {
      if (a.vec_s) {
        sx4 = ld_in<float4>(sxp + g, a.sx, static_cast<unsigned long long>(a.M) * a.KB);
        sw4 = ld_in<float4>(swp + g, a.sw, static_cast<unsigned long long>(a.NB) * a.KB);
      } else {
        const int g1 = min(g + 1, a.KB - 1), g2 = min(g + 2, a.KB - 1), g3 = min(g + 3, a.KB - 1);
        sx4 = make_float4(x1(g), x1(g1), x1(g2), x1(g3));
        sw4 = make_float4(w1(g), w1(g1), w1(g2), w1(g3));
      }
    };
    auto begin = [&](const Fp8Piece& q) {
      work.tile_at(q.tile, mt, nt);
      const int m = (mt * 2 + static_cast<int>(rank)) * kFp8Rows + row;
      const int nb = (nt * C::NT + half * C::kCols) / kFp8Block;
      sxp = a.sx + static_cast<size_t>(min(m, a.M - 1)) * a.KB;
      swp = a.sw + static_cast<size_t>(min(nb, a.NB - 1)) * a.KB;
      scales(q.k0 & ~3);
    };
    grid_dep_wait();
    Fp8Piece nx;
    bool have = work.next(nx);
    if (have) begin(nx);
    while (have) {
      p = nx;
      const int m0 = (mt * 2 + static_cast<int>(rank)) * kFp8Rows;
      const int rows = min(kFp8Rows, a.M - m0);  // may be <= 0 in a pair's second CTA
      const bool busy = quad * 32 < rows;
      const int ntile = nt, n0 = nt * C::NT + half * C::kCols;
      float acc[C::kCols];
#pragma unroll
      for (int j = 0; j < C::kCols; ++j) acc[j] = 0.0f;
      float f0 = 0.f, f1 = 0.f, f2 = 0.f, f3 = 0.f;  // scales of this block and the next ones
      auto next_four = [&](int g) {
        f0 = sx4.x * sw4.x;
        f1 = sx4.y * sw4.y;
        f2 = sx4.z * sw4.z;
        f3 = sx4.w * sw4.w;
        if (g + 4 < p.k1) scales(g + 4);
      };
      next_four(p.k0 & ~3);
      for (int i = 0; i < (p.k0 & 3); ++i) {
        f0 = f1;
        f1 = f2;
        f2 = f3;
      }
#pragma unroll 1
      for (int kb = p.k0; kb < p.k1; ++kb, ++it) {
        const float f = f0;
        const uint32_t b = it & (C::kBufs - 1);
        if (ok)
          ok = mbar_wait_warp(&tfull[b], (it / C::kBufs) & 1);
        else
          __syncwarp();  // the tensor-memory loads are of whole warps
        tc_fence_after();
        if (busy) {
          // the next 16 columns load while the last are added
          uint32_t v[2][16];
          tmem_ld16(taddr + b * C::NT, v[0]);
#pragma unroll
          for (int c = 0; c < C::kCols / 16; ++c) {
            tmem_wait_ld16(v[c & 1]);
            if (c + 1 < C::kCols / 16)
              tmem_ld16(taddr + b * C::NT + 16 * (c + 1), v[(c + 1) & 1]);
            else
              release(b);
#pragma unroll
            for (int j = 0; j < 16; j += 2)
              fma2(acc[16 * c + j], acc[16 * c + j + 1], f, v[c & 1][j], v[c & 1][j + 1]);
          }
        } else {
          release(b);
        }
        f0 = f1;
        f1 = f2;
        f2 = f3;
        if ((kb & 3) == 3 && kb + 1 < p.k1) next_four(kb + 1);
      }
      // the next piece's first scales travel while this one's sums are stored
      have = work.next(nx);
      if (have) begin(nx);
      if (p.k0 == 0 && p.k1 == a.KB) {
        if (!busy) continue;
        // through shared memory, 64 columns at a time: a thread's columns of its
        // token, 16 bytes at a time, swizzled so that 8 lanes' stores meet 8
        // different bank groups
#pragma unroll
        for (int h = 0; h < C::kCols / 64; ++h) {
          if (n0 + 64 * h >= a.N) break;
          if (lane == 0) bulk_wait_read();  // the last copy has left the box
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float* s8 = acc + 64 * h + 8 * c;
            uint4 o;
            o.x = bf16_pack2(s8[0], s8[1]);
            o.y = bf16_pack2(s8[2], s8[3]);
            o.z = bf16_pack2(s8[4], s8[5]);
            o.w = bf16_pack2(s8[6], s8[7]);
            *reinterpret_cast<uint4*>(yw + lane * 128 + ((c ^ (lane & 7)) << 4)) = o;
          }
          if (a.vec) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&ymap, yw, n0 + 64 * h, m0 + quad * 32, 0);
              bulk_commit();
            }
            __syncwarp();
          } else {
            __syncwarp();
            for (int r = 0; r < 32 && quad * 32 + r < rows; ++r) {
              uint16_t* y = a.Y + static_cast<size_t>(m0 + quad * 32 + r) * a.N + n0 + 64 * h;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int col = 32 * c + lane;
                if (n0 + 64 * h + col < a.N)
                  st_in(y + col, a.Y, static_cast<unsigned long long>(a.M) * a.N,
                        *reinterpret_cast<const uint16_t*>(yw + r * 128 + (((col >> 3) ^ (r & 7)) << 4) +
                                                           (col & 7) * 2));
              }
            }
            __syncwarp();
          }
        }
        continue;
      }
      // a run of the tail: publish the partial sums; the last run of the tile
      // to arrive adds them in the order of K
      const int tt = p.tile - a.rounds * a.workers;
      const int ubase = tt * a.KB;
      const int first = work.run_of(ubase), last = work.run_of(ubase + a.KB - 1);
      // a worker's run starts in this tile, or ends here after the one before
      constexpr size_t kSlot = static_cast<size_t>(kFp8Rows) * C::NT;
      auto slot_of = [&](int c) -> size_t {
        const size_t idx = work.run_start(c) < ubase ? 1 : 0;
        return ((static_cast<size_t>(c) * 2 + idx) * 2 + rank) * kSlot;
      };
      // a slot is [4 columns][token]: the lanes of a store are consecutive
      const size_t mine = slot_of(worker);
      if (row < rows && in_bounds(mine + kSlot - 1, a.partial_floats)) {
        float4* dst = reinterpret_cast<float4*>(a.partial + mine) + (half * C::kCols / 4) * kFp8Rows + row;
#pragma unroll
        for (int c = 0; c < C::kCols / 4; ++c)
          dst[c * kFp8Rows] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
      }
      epi_sync();
      if (threadIdx.x == 128) {
        bool is_last = false;
        if (in_bounds(static_cast<unsigned>(tt), a.tail)) {
          unsigned int* ctr = a.counter + tt * 2 + static_cast<int>(rank);
          // (the barrier and this acquire-release publish the CTA's sums and make
          // the other runs' visible)
          is_last = atom_add_acq_rel_gpu(ctr, 1u) == static_cast<unsigned>(last - first);
          if (is_last) *ctr = 0u;  // leave the workspace zeroed
        }
        *last_flag = is_last ? 1 : 0;
      }
      epi_sync();
      if (*last_flag) {
        const size_t s0 = slot_of(first);
        // runs after the first start inside this tile: their first slots
        const size_t s1 = (static_cast<size_t>(first) * 4 + rank) * kSlot;
        // a thread adds 8 columns of one token, kE such elements of two runs in
        // flight (16 loads per L2 round trip: the reading is latency-bound); the
        // additions stay in the order of the runs
        constexpr int kE = 4, kRuns = 2, kStep = kFp8EpiWarps * 32;
        const int tid = static_cast<int>(threadIdx.x) - 128;
#pragma unroll 1
        for (int e0 = tid; e0 < kFp8Rows * C::NT / 8; e0 += kE * kStep) {
          float4 sum[kE][2];
#pragma unroll
          for (int j = 0; j < kE; ++j) sum[j][0] = sum[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int c = first; c <= last; c += kRuns) {
            float4 v[kRuns][kE][2];
#pragma unroll
            for (int u = 0; u < kRuns; ++u) {
              const size_t slot = c + u == first ? s0 : s1 + static_cast<size_t>(c + u - first) * 4 * kSlot;
              const float4* src = reinterpret_cast<const float4*>(a.partial + slot);
#pragma unroll
              for (int j = 0; j < kE; ++j) {
                const int e = e0 + j * kStep;
                const int r = e % kFp8Rows, c8 = e / kFp8Rows;
                const bool live = c + u <= last && r < rows &&
                                  in_bounds(slot + kSlot - 1, a.partial_floats);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  v[u][j][h] = live ? __ldcg(src + (2 * c8 + h) * kFp8Rows + r)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
              }
            }
#pragma unroll
            for (int u = 0; u < kRuns; ++u) {
              if (c + u > last) break;
#pragma unroll
              for (int j = 0; j < kE; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  sum[j][h].x += v[u][j][h].x;
                  sum[j][h].y += v[u][j][h].y;
                  sum[j][h].z += v[u][j][h].z;
                  sum[j][h].w += v[u][j][h].w;
                }
            }
          }
#pragma unroll
          for (int j = 0; j < kE; ++j) {
            const int e = e0 + j * kStep;
            const int r = e % kFp8Rows, n = ntile * C::NT + e / kFp8Rows * 8;
            if (r >= rows) continue;
            uint16_t* y = a.Y + static_cast<size_t>(m0 + r) * a.N + n;
            const float o[8] = {sum[j][0].x, sum[j][0].y, sum[j][0].z, sum[j][0].w,
                                sum[j][1].x, sum[j][1].y, sum[j][1].z, sum[j][1].w};
            if (a.vec && n + 8 <= a.N) {
              st_in(y, a.Y, static_cast<unsigned long long>(a.M) * a.N,
                    make_uint4(bf16_pack2(o[0], o[1]), bf16_pack2(o[2], o[3]), bf16_pack2(o[4], o[5]),
                               bf16_pack2(o[6], o[7])));
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (n + i < a.N)
                  st_in(y + i, a.Y, static_cast<unsigned long long>(a.M) * a.N,
                        __bfloat16_as_ushort(__float2bfloat16_rn(o[i])));
            }
          }
        }
      }
    }
  }

  if (warp >= 4 && lane == 0) bulk_wait_all();  // output copies are complete
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may reach its memory
  if (warp == 1) {
    mbar_wait_warp(done, 0);  // every issued MMA has completed
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------- up to 128 tokens
// QUADS: tensor-memory lane quadrants in use (32 tokens each).  With fewer than
// 4 the MMA's other rows are whatever follows the token rows in shared memory
// (inside it: the weight stages), and their sums are never read.  Up to 64
// tokens two CTAs fit on an SM, so that the next call's set up and bring their
// first weights into L2 while this one's finish.
template <int QUADS_, int STAGES_>
struct Fp8RowsCfg {
  static constexpr int QUADS = QUADS_;
  static constexpr int STAGES = STAGES_;
  static constexpr int kXStage = QUADS * 32 * 128;
  static constexpr int kWStage = 128 * 128;
  // epilogue warps: those whose number modulo 4 is a used quadrant
  static constexpr int kWarps = QUADS == 1 ? 5 : QUADS == 2 ? 6 : 10;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kProducer = QUADS == 1 ? 1 : QUADS == 2 ? 2 : 8;
  static constexpr int kMma = kProducer + 1;
  static constexpr int kMinBlocks = QUADS == 4 ? 1 : 2;
  static constexpr int kEpiWarps = 2 * QUADS;
  // row stride of the fp32 sums in shared memory: 16 bytes past 128 columns,
  // so that 8 lanes' 16-byte stores of 8 rows meet different banks
  static constexpr int kRow = 132;
  static constexpr int kRing = STAGES * (kXStage + kWStage);
  static constexpr int kSmemBytes = 1024 + kRing + (2 * STAGES + 5) * 8 + 16;
  static_assert(QUADS * 32 * kRow * 4 <= kRing, "the sums reuse the ring");
  static_assert(STAGES * kWStage >= 128 * 128, "the MMA's unused rows stay inside");
  static_assert(kMinBlocks * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
};

// Scales of a thread's blocks in groups of four, requested one group ahead (the
// loads go to L2, 16 bytes where rows are aligned): f0..f3 are the scales of
// the current block and the next ones, shifted block by block.
struct Fp8Scales {
  float f0, f1, f2, f3;
  float4 x, w;  // the next group, as loaded
  // four of each, from arrays of nx elements from bx and nw from bw
  __device__ __forceinline__ void load4(const float* px, const float* bx, unsigned long long nx,
                                        const float* pw, const float* bw, unsigned long long nw) {
    x = ld_in<float4>(px, bx, nx);
    w = ld_in<float4>(pw, bw, nw);
  }
  __device__ __forceinline__ void take() {
    f0 = x.x * w.x;
    f1 = x.y * w.y;
    f2 = x.z * w.z;
    f3 = x.w * w.w;
  }
  __device__ __forceinline__ void shift() {
    f0 = f1;
    f1 = f2;
    f2 = f3;
  }
};

struct Fp8RowsArgs {
  const float* sx;  // [M, KB]
  const float* sw;  // [NB, KB]
  uint16_t* Y;      // bf16 [M, N]
  int M, N, KB;
  int splits;       // CTAs of a cluster: K ranges of a tile
  int vec_s;        // sx and sw rows are 16-byte aligned
  int vec;          // Y rows are 8-byte aligned
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kMinBlocks)
    fp8_rows_gemm_kernel(const __grid_constant__ CUtensorMap xmap,
                         const __grid_constant__ CUtensorMap wmap, const Fp8RowsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem;                         // STAGES x kXStage
  uint8_t* ws = xs + C::STAGES * C::kXStage;  // STAGES x kWStage
  float* sums = reinterpret_cast<float*>(smem);  // [tokens][kRow], once the ring is idle
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);  // landed (tx)
  uint64_t* empty = full + C::STAGES;         // MMAs done reading (commit)
  uint64_t* tfull = empty + C::STAGES;        // block sum ready (commit)   [2]
  uint64_t* tempty = tfull + 2;               // block sum read (epilogue)  [2]
  uint64_t* done = tempty + 2;                // every MMA complete (commit)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nt = static_cast<int>(blockIdx.x) / a.splits;
  const int rank = static_cast<int>(blockIdx.x) - nt * a.splits;  // the cluster's CTAs in order
  const int k0 = static_cast<int>(static_cast<long long>(a.KB) * rank / a.splits);
  const int k1 = static_cast<int>(static_cast<long long>(a.KB) * (rank + 1) / a.splits);
  const int n = k1 - k0;

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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool epi = (warp & 3) < C::QUADS && warp < 8;

  if (warp == C::kProducer) {
    if (lane == 0) {
      prefetch_tensormap(&wmap);
      prefetch_tensormap(&xmap);
      const uint64_t pol_w = policy_evict_first();  // read once
      const uint64_t pol_x = policy_evict_last();
      const uint32_t bytes = C::kWStage + static_cast<uint32_t>(a.M) * 128u;
      // the first ring of weights into L2 ahead of the dependency wait, as in the
      // pair kernel (1 x 4096 x 4096 in a chain of products 7.3 us, without it
      // 7.7; four rings 7.7, they displace each other.  Weights read ahead of
      // the wait, out of the stream's order, were 6.8)
      for (int i = 0; i < n && i < C::STAGES; ++i)
        tma_prefetch_3d(&wmap, (k0 + i) * 128, nt * 128, 0, pol_w);
      grid_dep_wait();
      int i = 0;
      for (; i < n; ++i) {
        const int s = i % C::STAGES;
        if (i >= C::STAGES && !mbar_wait(&empty[s], ((i / C::STAGES) - 1) & 1)) break;
        mbar_arrive_expect_tx(&full[s], bytes);
        tma_load_3d(ws + s * C::kWStage, &wmap, (k0 + i) * 128, nt * 128, 0, &full[s], pol_w);
        tma_load_3d(xs + s * C::kXStage, &xmap, (k0 + i) * 128, 0, 0, &full[s], pol_x);
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
      // descriptor addresses are in units of 16 bytes
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
  } else if (epi) {
    const int quad = warp & 3, half = warp >> 2;
    const int row = quad * 32 + lane;
    const bool busy = quad * 32 < a.M;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 64;
    const uint32_t te0 = smem_u32(&tempty[0]);
    const float* sxp = a.sx + static_cast<size_t>(min(row, a.M - 1)) * a.KB + k0;
    const float* swp = a.sw + static_cast<size_t>(nt) * a.KB + k0;
    float acc[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) acc[j] = 0.0f;
    bool ok = true;  // after a wait gave up: go through the motions without waiting
    Fp8Scales sc;
    // aligned rows: groups of the row's own fours; else from the first block on
    const int ph = a.vec_s ? k0 & 3 : 0;
    const unsigned long long n_sx = static_cast<unsigned long long>(a.M) * a.KB;
    const unsigned long long n_sw = static_cast<unsigned long long>((a.N + 127) / 128) * a.KB;
    const auto x1 = [&](int i) { return ld_in<float>(sxp + i, a.sx, n_sx); };
    const auto w1 = [&](int i) { return ld_in<float>(swp + i, a.sw, n_sw); };
    auto request = [&](int i) {  // the group that starts with block i of this range
      if (a.vec_s) {
        sc.load4(sxp + i, a.sx, n_sx, swp + i, a.sw, n_sw);
      } else {
        const int i1 = min(i + 1, n - 1), i2 = min(i + 2, n - 1), i3 = min(i + 3, n - 1);
        sc.x = make_float4(x1(i), x1(i1), x1(i2), x1(i3));
        sc.w = make_float4(w1(i), w1(i1), w1(i2), w1(i3));
      }
    };
    grid_dep_wait();
    request(-ph);
    sc.take();
    if (4 - ph < n) request(4 - ph);
    for (int j = 0; j < ph; ++j) sc.shift();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int b = i & 1;
      if (i > 0 && ((i + ph) & 3) == 0) {
        sc.take();
        if (i + 4 < n) request(i + 4);
      }
      const float f = sc.f0;
      sc.shift();
      if (ok)
        ok = mbar_wait_warp(&tfull[b], (i >> 1) & 1);
      else
        __syncwarp();  // the tensor-memory loads are of whole warps
      tc_fence_after();
      if (busy) {
        // the buffer goes back as soon as its columns are in registers: the
        // round trip from MMA to MMA bounds a CTA's rate
        uint32_t v0[32], v1[32];
        tmem_ld64_wait(taddr + b * 128, v0, v1);
        tc_fence_before();
        mbar_arrive_lane0(te0 + 8 * b, lane);
#pragma unroll
        for (int j = 0; j < 32; j += 2) fma2(acc[j], acc[j + 1], f, v0[j], v0[j + 1]);
#pragma unroll
        for (int j = 0; j < 32; j += 2) fma2(acc[32 + j], acc[33 + j], f, v1[j], v1[j + 1]);
      } else {
        tc_fence_before();
        mbar_arrive_lane0(te0 + 8 * b, lane);
      }
    }
    // every MMA of this CTA has read its operands (the last block's sum is
    // complete), so the ring takes the sums
    if (ok && row < a.M) {
      float* dst = sums + row * C::kRow + half * 64;
#pragma unroll
      for (int c = 0; c < 16; ++c)
        *reinterpret_cast<float4*>(dst + 4 * c) =
            make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
    }
  }
  __syncwarp();
  tc_fence_before();
  // the cluster's sums are in place (a single CTA: its own)
  if (a.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  // each CTA adds its share of the columns over the K ranges, in order of K
  {
    const int q0 = 32 * rank / a.splits, q1 = 32 * (rank + 1) / a.splits;  // in units of 4 columns
    const int w = q1 - q0;
    const uint32_t mine = smem_u32(sums);
    for (int e = threadIdx.x; e < a.M * w; e += C::kThreads) {
      const int r = e / w, c = (q0 + e - r * w) * 4;
      const uint32_t at = mine + static_cast<uint32_t>(r * C::kRow + c) * 4u;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.splits == 1) {
        sum = *reinterpret_cast<const float4*>(sums + r * C::kRow + c);
      } else {
        float4 v[8];
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p < a.splits) v[p] = ld_cluster_f4(mapa_shared(at, p));
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p < a.splits) {
            sum.x += v[p].x;
            sum.y += v[p].y;
            sum.z += v[p].z;
            sum.w += v[p].w;
          }
      }
      const int col = nt * 128 + c;
      uint16_t* y = a.Y + static_cast<size_t>(r) * a.N + col;
      const unsigned long long n_y = static_cast<unsigned long long>(a.M) * a.N;
      if (a.vec && col + 4 <= a.N) {
        st_in(y, a.Y, n_y, make_uint2(bf16_pack2(sum.x, sum.y), bf16_pack2(sum.z, sum.w)));
      } else {
        const float s4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < a.N) st_in(y + j, a.Y, n_y, __bfloat16_as_ushort(__float2bfloat16_rn(s4[j])));
      }
    }
  }
  if (a.splits > 1)
    cluster_sync();  // no CTA leaves while another reads its sums
  else
    __syncthreads();
  if (warp == C::kMma) {
    mbar_wait_warp(done, 0);  // every issued MMA has completed
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace w4
