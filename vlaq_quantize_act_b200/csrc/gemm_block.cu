// FP8 E4M3 GEMM with block scales of 128 on the sm_100a tensor cores.
//
//   Y[m, n] = bf16_rne( sum_b s_x[b, m] s_w[n / 128, b] P_b[m, n] + residual[m, n] )
//   P_b[m, n] = sum_{k in block b} e4m3(x[m, k]) e4m3(w[n, k])
//
// The fp32 scales cannot go into the MMA (its block scales are powers of two
// or E4M3), so each block of 128 along K is one accumulation of its own in
// TMEM (four MMAs of K = 32), and epilogue warps add it, scaled, to fp32 sums
// that stay in their registers: acc = fma(P_b, s_x s_w, acc).  One
// accumulator buffer is read while the next block's MMAs fill another.
//   gemm_block_pair_kernel  256 x 256 tiles over the two CTAs of a cluster
//                           (paired MMA), token rows on the TMEM lanes: one
//                           scale per thread and block; or over two pairs
//                           that take half of K each.
//   gemm_block_rows_kernel  128 tokens x 128 weight rows per CTA, token rows on
//                           the lanes, K split over the CTAs of a cluster when
//                           the tiles are few; more than 64 tokens whose
//                           256 x 256 tiles would leave SMs idle.
//   gemm_block_cols_kernel  128 weight rows on the TMEM lanes and 16, 32 or 64
//                           token columns: a decode step's tile is as narrow
//                           as its tokens, and the tile reads each weight
//                           once; K split like that.
// The CTAs of a cluster add their sums over each other's shared memory, in the
// order of K: no workspace and the same result every time.
//
// Times are device times of a call, in a CUDA graph of calls over buffers larger
// than L2, where nothing else is said; a pair of times with an arrow is one
// change, measured before and after it.
//
// Every mbarrier wait is bounded (clock budget); a wait that runs out sets a
// shared abort flag and the device status word, and the roles stop.  Once all of
// them have, a CTA that gave up stays until its copies in flight have landed
// (let_copies_land), frees its TMEM and returns.  Tiles that were given up are
// not stored, or, where a cluster of the rows and columns kernels adds the sums
// of its CTAs, stored as NaN: the flags of the other CTAs cost 0.1 to 0.3 us of
// every call to ask for.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"
#include "tensor_map.h"

namespace vlaq {

__device__ unsigned int g_vlaq_block_status = 0;

namespace {

constexpr int kTmemColumns = 512;
constexpr int kRowBytes = 128;              // one block of 128 codes of a row
constexpr int kTileBytes = 128 * kRowBytes;  // 128 rows of it
constexpr int kPrefetchBlocks = 4;           // weight blocks brought into L2 before the dependency wait

struct BlockArgs {
  const float* sx;  // [blocks][M]
  const float* sw;  // [ceil(N / 128)][blocks]
  const __nv_bfloat16* residual;
  __nv_bfloat16* Y;
  int M, N;
  int blocks;       // ceil(K / 128)
  int m_tiles, n_tiles, units;
  long long budget;
};

__device__ __forceinline__ void give_up(volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(&g_vlaq_block_status, kStatusTimeout);
}

// Bounded wait that also gives up once another role (or, in a pair, a role of
// the other CTA: peer_abort != 0) aborted.  The wait sleeps in the barrier
// unit: polling it cost 225 W of the GPU's 1000 W, which its clock pays for
// (4580 x 3584 x 18944: 417 -> 411 us).
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, long long budget,
                                             volatile int* abort_flag, uint32_t peer_abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait_long(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > budget) {
      give_up(abort_flag);
      if (peer_abort) st_shared_cluster_u32(peer_abort, 1u);
      return false;
    }
  }
}

// The same by all lanes of a warp, which leave together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long budget, volatile int* abort_flag,
                                          uint32_t peer_abort) {
  return __all_sync(0xffffffffu, bounded_wait(bar, parity, budget, abort_flag, peer_abort));
}

// A thread's n sums of a tile that was given up, for the CTAs that add them:
// not numbers, once no copy writes over them any more.
__device__ __noinline__ void give_up_sums(float* sums, int n, int stride) {
  let_copies_land();
  for (int j = 0; j < n; ++j) sums[j * stride] = __int_as_float(0x7FFFFFFF);
}

// Values computed here, not where they are first used.
__device__ __forceinline__ void keep(int a, int b, int c) { asm volatile("" ::"r"(a), "r"(b), "r"(c) : "memory"); }

// acc[j] += p[j] s for 32 columns, two per instruction.
__device__ __forceinline__ void add_scaled32(float* acc, const uint32_t (&p)[32], float s) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float2 r = __ffma2_rn(make_float2(__uint_as_float(p[j]), __uint_as_float(p[j + 1])), make_float2(s, s),
                                make_float2(acc[j], acc[j + 1]));
    acc[j] = r.x;
    acc[j + 1] = r.y;
  }
}

// Scales s_x s_w of n consecutive blocks for an epilogue thread's row and
// weight block.  The row's scales come through the thread's own ring of four
// slots in shared memory, copied four blocks ahead (a load into a register
// makes the warp wait for it where the register moves on: with the next
// block's scale in a register every block took an L2 round trip), the
// weight's 32 blocks at a time, one per lane.
constexpr int kScaleSlots = 4;
template <int THREADS>  // epilogue threads: distance of a thread's slots
struct ScaleStream {
  const float* sx;  // the row's scale of block 0; M apart from the next
  const float* sw;
  int n;
  float* slots;
  float w, w_next;

  __device__ __forceinline__ void copy(int i, int M) {
    if (i < n) cp_async4(smem_u32(slots + (i % kScaleSlots) * THREADS), sx + static_cast<int64_t>(i) * M);
    cp_async_commit();
  }
  __device__ __forceinline__ void start(const float* row_scales, const float* weight_scales, int blocks,
                                        float* thread_slots, int M, int lane) {
    sx = row_scales;
    sw = weight_scales;
    n = blocks;
    slots = thread_slots;
    w_next = __ldg(sw + min(lane, n - 1));
#pragma unroll
    for (int i = 0; i < kScaleSlots; ++i) copy(i, M);
  }
  // The scale of block i; called for i = 0, 1, ...
  __device__ __forceinline__ float next(int i, int M, int lane) {
    if ((i & 31) == 0) {
      w = w_next;
      w_next = __ldg(sw + min(i + 32 + lane, n - 1));
    }
    cp_async_wait<kScaleSlots - 1>();
    const float s = slots[(i % kScaleSlots) * THREADS] * __shfl_sync(0xffffffffu, w, i & 31);
    copy(i + kScaleSlots, M);
    return s;
  }
};

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Barrier over the epilogue warps (`threads` threads).  All of them reach it
// the same number of times whatever happens: a warp whose wait ran out skips
// its work, not its barriers.
__device__ __forceinline__ void epilogue_sync(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

// Y[m, n .. n + 3] = bf16(y + residual).
__device__ __forceinline__ void store4(const BlockArgs& a, float4 y, int m, int n) {
  const size_t o = static_cast<size_t>(m) * a.N + n;
  if (a.residual) {
    const uint2 rv = *reinterpret_cast<const uint2*>(a.residual + o);
    y.x += __uint_as_float(rv.x << 16);
    y.y += __uint_as_float(rv.x & 0xFFFF0000u);
    y.z += __uint_as_float(rv.y << 16);
    y.w += __uint_as_float(rv.y & 0xFFFF0000u);
  }
  *reinterpret_cast<uint2*>(a.Y + o) = make_uint2(bf16x2(y.x, y.y), bf16x2(y.z, y.w));
}

// y += v.
__device__ __forceinline__ void add4(float4& y, const float4& v) {
  y.x += v.x;
  y.y += v.y;
  y.z += v.z;
  y.w += v.w;
}

// Sums of the rows kernel's clusters: rows of 128 fp32 columns, 16-byte
// groups permuted by the row and their halves swapped in rows 8 .. 15 mod 16,
// so that a half warp's 8-byte writes, one row per lane, fall on all banks.
// (Written 8 bytes at a time here and in the pair kernel: 16-byte stores tie
// the sums to groups of four registers, and the multiply-adds of the loop
// before took longer: 480 -> 600 ns for a block of the pair kernel, 50 -> 52 us
// for 512 x 3584 x 18944 in the rows kernel.)
constexpr int kSumRowBytes = 128 * 4;
__device__ __forceinline__ uint32_t sum_offset(int row, int group) {
  return static_cast<uint32_t>(row * kSumRowBytes + ((group ^ (row & 7)) << 4));
}
template <int COLS>
__device__ __forceinline__ void write_sums(uint32_t base, int row, const float (&acc)[COLS], int group0 = 0) {
  const uint32_t swap = static_cast<uint32_t>(row & 8);
#pragma unroll
  for (int c = 0; c < COLS; c += 4) {
    const uint32_t at = base + sum_offset(row, group0 + c / 4);
    st_shared_f2(at + swap, acc[c], acc[c + 1]);
    st_shared_f2(at + (swap ^ 8u), acc[c + 2], acc[c + 3]);
  }
}
// Four columns of a row in the CTA with that base.
__device__ __forceinline__ float4 read_sums(uint32_t base, int row, int group) {
  const float4 v = ld_shared_cluster_f4(base + sum_offset(row, group));
  return row & 8 ? make_float4(v.z, v.w, v.x, v.y) : v;
}

// ---------------------------------------------------------------------------
// CTA r of a pair loads rows [128 r, 128 r + 128) of the x tile and of the w
// tile; the paired MMA gives it the 128 x 256 accumulator of its own rows.
// Two 256-column accumulator buffers fill TMEM; block i uses buffer i % 2.
// One barrier pair per stage carries everything the MMA thread waits for: the
// leader's full barrier of block i completes on both CTAs' operand bytes and
// on the 16 epilogue warps that have read block i - 2 out of its buffer, and
// one commit per block to both CTAs' done barrier tells the producers that the
// stage is free and the epilogue warps that the block's sums are there.
//   warps 0, 2: producers of x and w; warp 1: TMEM allocator (both) and MMA
//   issuer (leader); warp 3: idle; warps 4-11: epilogue, warp e = w - 4 has
//   TMEM lanes 32 (w % 4) .. + 31 (its token rows) and columns 128 (e / 4) ..
//   + 127 (one weight scale per block).
// The sums take 128 registers per epilogue thread: warps 0-3 give theirs up
// (40), warps 4-11 take 232: 40 + 2 * 232 = 3 * 168 (the build checks that
// ptxas allocates 168 at entry).
//
// What bounds it: the board's 1000 W.  In a loop of seconds 1024 x 37888 x 3584
// takes 153 us (1.82 PFLOP/s) at 1.38 GHz, 4580 x 3584 x 18944 357 us (1.74) at
// 1.43 GHz (a first few calls, before the power limit acts, 133 and 314 us); the
// per-row FP8 kernel, whose sums stay in TMEM, 132 and 299 us at 1.31 GHz, and
// this kernel without its epilogue 285 us.  A block takes about 850 clocks of
// which the MMA is 512: the rest is the round trip from commit to the epilogue
// warps and back (about 420 clocks by itself) and the 32768 products of a
// block (281 clocks of the SM's packed multiply-add pipe), less what two
// buffers overlap.  Measured against this split: 16 epilogue warps of 64
// columns 172 / 380 us (more instructions per product), MMAs of 128 columns
// with a barrier for each half 170 / 399 us (twice the round trips).
//
// SPLIT: few tiles and a long K.  A cluster of two pairs has one tile, each pair
// half of its blocks; then each CTA sends the sums of half of its columns to
// the other pair's CTA of its rows and stores the other half.  512 x 3584 x
// 18944 (28 tiles): 64 -> 41 us; the exchange and the start of the larger
// cluster cost about 3 us (reads of the other CTA's sums one row per lane, not
// side by side: 8 us).
struct PairTile {
  static constexpr int BM = 256, BN = 256;
  static constexpr int STAGE_BYTES = 2 * kTileBytes;
  static constexpr int STAGES = 4;
  static constexpr int EPI_WARPS = 8;
  static constexpr int COLS = BN / (EPI_WARPS / 4);  // columns of an epilogue warp
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int REGS_ROLES = 40, REGS_EPI = 232;
  static_assert(REGS_ROLES + EPI_WARPS / 4 * REGS_EPI == (1 + EPI_WARPS / 4) * 168, "register split");
  static constexpr int OUT_BYTES = 32 * 128;         // 32 rows x 64 bf16 columns of an epilogue warp
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_WARPS * 2 * OUT_BYTES + 1024;
  // kind::f8f6f4, E4M3 x E4M3, fp32 accumulator, N = 256, M = 256
  static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(BM >> 4) << 24);
  static_assert(128 * COLS * 4 <= STAGES * STAGE_BYTES, "half of a CTA's sums fit its stages");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

template <bool SPLIT>
__global__ void __launch_bounds__(PairTile::THREADS, 1)
gemm_block_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmR,
                       const BlockArgs a) {
  using C = PairTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];  // leader: operands of both CTAs, buffer read
  __shared__ __align__(8) uint64_t done_bar[C::STAGES];  // block accumulated (leader's commit)
  __shared__ __align__(8) uint64_t res_bar[C::EPI_WARPS];  // residual of the warp's part of the tile
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ float s_sx[kScaleSlots][32 * C::EPI_WARPS];  // each epilogue thread's own copies of its row's scales
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const uint32_t rank = cta & 1u;  // in the pair
  // SPLIT: a cluster of two pairs has one tile, pair `split` half of its blocks
  const int split = SPLIT ? static_cast<int>(cta >> 1) : 0;
  const int pair = static_cast<int>(blockIdx.x >> (SPLIT ? 2 : 1));
  const int pairs = static_cast<int>(gridDim.x >> 1);
  const int units = SPLIT ? pair + 1 : a.units;
  const int kb0 = SPLIT && split ? a.blocks >> 1 : 0;
  const int kb1 = SPLIT && !split ? a.blocks >> 1 : a.blocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full_bar[i], 1 + 2 * C::EPI_WARPS);
      mbar_init(&done_bar[i], 1);
    }
    for (int i = 0; i < C::EPI_WARPS; ++i) mbar_init(&res_bar[i], 1);
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmY);
    if (a.residual) prefetch_tensormap(&tmR);
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem_base, kTmemColumns);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs' barriers are initialised before either CTA signals the other's
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int*>(&s_abort)), cta ^ 1u);
  const uint32_t leader_full = mapa_shared(smem_u32(full_bar), cta & ~1u);
  const int first = (pair / a.m_tiles) * C::BN + 128 * static_cast<int>(rank);  // weight row of the first tile
  keep(kb0, kb1, first);                                                       // computed before the wait
  if (warp == 2 && elect_one())
    for (int b = kb0; b < min(kb1, kb0 + kPrefetchBlocks); ++b) tma_prefetch_2d(&tmW, b * kRowBytes, first);
  griddep_wait();
  griddep_launch_dependents();

  if (warp < 4) {
    regs_dec<C::REGS_ROLES>();
    if ((warp == 0 || warp == 2) && elect_one()) {
      // ---------------------------------------- producers (both CTAs): x, w
      const bool is_x = warp == 0;
      const CUtensorMap* map = is_x ? &tmX : &tmW;
      uint8_t* dst = smem + (is_x ? 0 : kTileBytes);
      int it = 0, stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const int row0 = (is_x ? (u % a.m_tiles) * C::BM : (u / a.m_tiles) * C::BN) + 128 * static_cast<int>(rank);
        for (int b = kb0; b < kb1; ++b, ++it) {
          if (it >= C::STAGES && !bounded_wait(&done_bar[stage], phase ^ 1u, a.budget, &s_abort, peer_abort)) {
            ok = false;
            break;
          }
          if (is_x && rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * C::STAGE_BYTES);
          tma_load_2d_pair(dst + stage * C::STAGE_BYTES, map, leader_full + 8u * stage, b * kRowBytes, row0);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the leader's last commits have landed in this CTA (unless a wait gives up)
      for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it && ok; ++i)
        ok = bounded_wait(&done_bar[i % C::STAGES], static_cast<uint32_t>(i / C::STAGES) & 1u, a.budget, &s_abort,
                          peer_abort);
    } else if (warp == 1 && rank == 0 && elect_one()) {
      // ------------------------------------------------- MMA issuer (leader)
      const uint64_t xd = sdesc_kmajor_sw128(smem_u32(smem)), wd = sdesc_kmajor_sw128(smem_u32(smem) + kTileBytes);
      int stage = 0;
      uint32_t phase = 0, buf = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        for (int b = kb0; b < kb1; ++b) {
          if (!bounded_wait(&full_bar[stage], phase, a.budget, &s_abort, peer_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(stage) * (C::STAGE_BYTES >> 4);  // descriptor units of 16 bytes
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f8f6f4_pair(tmem + buf, xd + off + 2 * j, wd + off + 2 * j, C::IDESC, j > 0);
          umma_commit_pair(&done_bar[stage], static_cast<uint16_t>(0x3u << cta));
          buf ^= C::BN;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      umma_commit_pair(&drain_bar, static_cast<uint16_t>(0x1u << cta));
      const long long t0 = clock64();
      while (!mbar_try_wait(&drain_bar, 0) && clock64() - t0 < 4 * a.budget + 1000000) {
      }
    }
  } else {
    // ------------------------------------------------- epilogue (both CTAs)
    regs_inc<C::REGS_EPI>();
    const int q = warp & 3;
    const int h = (warp - 4) >> 2;
    auto buffer_read = [&](int stage) {  // this warp has read the buffer that the block of that stage reuses
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(leader_full + 8u * stage);
    };
    buffer_read(0);
    buffer_read(1);
    const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(C::COLS * h);
    uint8_t* out = smem + C::STAGES * C::STAGE_BYTES + (warp - 4) * 2 * C::OUT_BYTES;
    uint32_t res_phase = 0;
    int stage = 0;
    float* slots = &s_sx[0][threadIdx.x - 128];
    uint32_t phase = 0, buf = 0;
    bool ok = true;
    for (int u = pair; u < units && ok; u += pairs) {
      const int row0 = (u % a.m_tiles) * C::BM + 128 * static_cast<int>(rank) + 32 * q;
      const int col0 = (u / a.m_tiles) * C::BN + C::COLS * h;
      const bool live = row0 < a.M && col0 < a.N;  // warp-uniform
      const bool stores = !SPLIT || h == split;  // this warp's columns are this CTA's to store
      if (a.residual && stores && lane == 0) {
        // the residual lands in the staging buffer while the blocks are summed;
        // the previous tile's stores have read it by then
        bulk_wait_group_read0();
        mbar_arrive_expect_tx(&res_bar[warp - 4], 2 * C::OUT_BYTES);
        tma_load_2d(out, &tmR, &res_bar[warp - 4], col0, row0);
        tma_load_2d(out + C::OUT_BYTES, &tmR, &res_bar[warp - 4], col0 + 64, row0);
      }
      // rows and columns past the output use the last ones' scales and are not stored
      ScaleStream<32 * C::EPI_WARPS> scales;
      scales.start(a.sx + static_cast<int64_t>(kb0) * a.M + min(row0 + lane, a.M - 1),
                   a.sw + static_cast<int64_t>(min(col0, a.N - 1) >> 7) * a.blocks + kb0, kb1 - kb0, slots, a.M, lane);
      float acc[C::COLS];
#pragma unroll
      for (int j = 0; j < C::COLS; ++j) acc[j] = 0.0f;
      for (int b = 0; b < kb1 - kb0; ++b) {
        const float sc = scales.next(b, a.M, lane);
        if (!warp_wait(&done_bar[stage], phase, a.budget, &s_abort, peer_abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::COLS; c += 32) {
          uint32_t p[32];
          tmem_ld_32x32b_x32(tbase + buf + c, p);
          tmem_ld_wait();
          if (c + 32 == C::COLS) buffer_read(stage + 2 < C::STAGES ? stage + 2 : stage + 2 - C::STAGES);
          add_scaled32(acc + c, p, sc);
        }
        buf ^= C::BN;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (SPLIT) {
        // Each CTA stores half of its rows' columns: the other half's sums go
        // through the stages (all loads have landed and all MMAs have read
        // them: the last block is done) to the CTA of the other pair.
        // Two columns of all lanes side by side, which is how they are read.
        const uint32_t sums = smem_u32(smem) + q * (32 * C::COLS * 4) + lane * 8;
        if (ok && !stores) {
#pragma unroll
          for (int c = 0; c < C::COLS; c += 2) st_shared_f2(sums + c * 128, acc[c], acc[c + 1]);
        }
        __syncwarp();
        cluster_sync();
        if (!stores) break;
        if (ok) {
          const uint32_t gave_up =
              ld_shared_cluster_u32(mapa_shared(smem_u32(const_cast<const int*>(&s_abort)), cta ^ 2u));
          const uint32_t other = mapa_shared(sums, cta ^ 2u);
#pragma unroll
          for (int c = 0; c < C::COLS; c += 2) {
            const float2 v = ld_shared_cluster_f2(other + c * 128);
            acc[c] += v.x;
            acc[c + 1] += v.y;
          }
          ok = __all_sync(0xffffffffu, gave_up == 0);
        }
      }
      if (!ok) break;
      // + residual, bf16, through the staging buffer (128-byte rows in the
      // copy engine's 128-byte swizzle) and out by tile stores, which clip
      // rows and columns past the output; the next tile's sums start meanwhile
      if (a.residual) {
        if (!warp_wait(&res_bar[warp - 4], res_phase, a.budget, &s_abort, peer_abort)) break;
        res_phase ^= 1u;
      } else {
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
      }
#pragma unroll
      for (int c = 0; c < C::COLS; c += 8) {
        const uint32_t at = smem_u32(out) + (c / 64) * C::OUT_BYTES + lane * 128 + ((((c / 8) & 7) ^ (lane & 7)) << 4);
        if (a.residual) {
          const uint4 rv = ld_shared_v4(at);
          const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[c + 2 * j] += __uint_as_float(rw[j] << 16);
            acc[c + 2 * j + 1] += __uint_as_float(rw[j] & 0xFFFF0000u);
          }
        }
        st_shared_v4(at, bf16x2(acc[c], acc[c + 1]), bf16x2(acc[c + 2], acc[c + 3]), bf16x2(acc[c + 4], acc[c + 5]),
                     bf16x2(acc[c + 6], acc[c + 7]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && live) {
        tma_store_2d(&tmY, out, col0, row0);
        if (col0 + 64 < a.N) tma_store_2d(&tmY, out + C::OUT_BYTES, col0 + 64, row0);
        bulk_commit_group();
      }
    }
    if (lane == 0) bulk_wait_group0();
  }

  // No CTA leaves (or frees its TMEM) while another may still signal it, read
  // its sums, or the paired MMAs may still touch its shared memory or TMEM.
  tc_fence_before();
  __syncwarp();
  if (SPLIT && warp < 4) cluster_sync_relaxed();  // (the epilogue warps' exchange of sums)
  cluster_sync();
  if (s_abort) let_copies_land();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemColumns);
  }
}

// ---------------------------------------------------------------------------
// One CTA per tile of 128 tokens (TMEM lanes) x 128 weight rows (columns), or
// a cluster of CTAs that take consecutive ranges of the tile's blocks and add
// their sums in shared memory; a cluster of one loops over tiles.
//   warps 0, 2: producers of x and w; warp 1: TMEM allocator and MMA issuer;
//   warp 3: idle; warps 4-11: epilogue, warp e = w - 4 has tokens 32 (w % 4)
//   .. + 31 and columns 64 (e / 4) .. + 63.
// Four accumulator buffers of 128 columns, block i in buffer i % 4; as in the
// pair kernel the full barrier of block i also waits for the epilogue warps
// that have read block i - 4.
//
// What bounds it: a block takes about 310 ns (600 clocks) in a long K, of which
// shared memory takes 512: 32 KB in by TMA and 32 KB out to the MMA, whose own
// time is 256.  512 x 3584 x 3584: 12.4 us (112 tiles), 128 x 3584 x 3584 8.5
// (28 tiles of four CTAs, HBM and the first stage), 333 x 1000 x 2000 7.2 (four).
// Measured against it: epilogue warps in two sets that take alternate blocks,
// 128 columns each, the same within 3%; four stages 12.5 us, prefetching
// weights 6 or 12 blocks ahead 13.1.
struct RowsTile {
  static constexpr int BM = 128, BN = 128;
  static constexpr int STAGE_BYTES = 2 * kTileBytes;
  static constexpr int STAGES = 5;
  static constexpr int BUFS = 4;
  static constexpr int EPI_WARPS = 8;
  static constexpr int COLS = BN / (EPI_WARPS / 4);
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int OUT_BYTES = 32 * 128;  // 32 rows x 64 bf16 columns of an epilogue warp
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_WARPS * OUT_BYTES + 1024;
  // kind::f8f6f4, E4M3 x E4M3, fp32 accumulator, N = 128, M = 128
  static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(BM >> 4) << 24);
  static_assert(BM * BN * 4 <= STAGES * STAGE_BYTES, "the cluster's sums fit the operand ring");
  static_assert(BUFS * BN <= kTmemColumns, "TMEM budget");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

__global__ void __launch_bounds__(RowsTile::THREADS, 1)
gemm_block_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmR,
                       const BlockArgs a, const int splits) {
  using C = RowsTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];    // operands of a block, buffer read
  __shared__ __align__(8) uint64_t done_bar[C::STAGES];    // block accumulated
  __shared__ __align__(8) uint64_t res_bar[C::EPI_WARPS];  // residual of the warp's part of the tile
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ float s_sx[kScaleSlots][32 * C::EPI_WARPS];  // each epilogue thread's own copies of its row's scales
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int group = static_cast<int>(blockIdx.x) / splits;
  const int groups = static_cast<int>(gridDim.x) / splits;
  // blocks <= 2^24, splits <= 8
  const int kb0 = static_cast<int>(static_cast<uint32_t>(a.blocks * rank) / static_cast<uint32_t>(splits));
  const int kb1 = static_cast<int>(static_cast<uint32_t>(a.blocks * (rank + 1)) / static_cast<uint32_t>(splits));

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full_bar[i], 1 + C::EPI_WARPS);
      mbar_init(&done_bar[i], 1);
    }
    for (int i = 0; i < C::EPI_WARPS; ++i) mbar_init(&res_bar[i], 1);
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmY);
    if (a.residual) prefetch_tensormap(&tmR);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem_base, C::BUFS * C::BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  const int first = (group / a.m_tiles) * C::BN;  // weight row of the first tile
  keep(kb0, kb1, first);                          // computed before the wait
  if (warp == 2 && elect_one())
    for (int b = kb0; b < min(kb1, kb0 + kPrefetchBlocks); ++b) tma_prefetch_2d(&tmW, b * kRowBytes, first);
  griddep_wait();
  griddep_launch_dependents();

  if ((warp == 0 || warp == 2) && elect_one()) {
    // ----------------------------------------------------- producers: x, w
    const bool is_x = warp == 0;
    const CUtensorMap* map = is_x ? &tmX : &tmW;
    uint8_t* dst = smem + (is_x ? 0 : kTileBytes);
    int it = 0, stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = group; u < a.units && ok; u += groups) {
      const int row0 = is_x ? (u % a.m_tiles) * C::BM : (u / a.m_tiles) * C::BN;
      for (int b = kb0; b < kb1; ++b, ++it) {
        if (it >= C::STAGES && !bounded_wait(&done_bar[stage], phase ^ 1u, a.budget, &s_abort, 0)) {
          ok = false;
          break;
        }
        if (is_x) mbar_arrive_expect_tx(&full_bar[stage], C::STAGE_BYTES);
        tma_load_2d(dst + stage * C::STAGE_BYTES, map, &full_bar[stage], b * kRowBytes, row0);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1 && elect_one()) {
    // ----------------------------------------------------------- MMA issuer
    const uint64_t xd = sdesc_kmajor_sw128(smem_u32(smem)), wd = sdesc_kmajor_sw128(smem_u32(smem) + kTileBytes);
    int stage = 0;
    uint32_t phase = 0, buf = 0;
    bool ok = true;
    for (int u = group; u < a.units && ok; u += groups) {
      for (int b = kb0; b < kb1; ++b) {
        if (!bounded_wait(&full_bar[stage], phase, a.budget, &s_abort, 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(stage) * (C::STAGE_BYTES >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f8f6f4(tmem + buf, xd + off + 2 * j, wd + off + 2 * j, C::IDESC, j > 0);
        umma_commit(&done_bar[stage]);
        buf = (buf + C::BN) & (C::BUFS * C::BN - 1);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    umma_commit(&drain_bar);
    const long long t0 = clock64();
    while (!mbar_try_wait(&drain_bar, 0) && clock64() - t0 < 4 * a.budget + 1000000) {
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int h = (warp - 4) >> 2;
    auto buffer_read = [&](int stage) {  // this warp has read the buffer that the block of that stage reuses
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(&full_bar[stage]);
    };
#pragma unroll
    for (int i = 0; i < C::BUFS; ++i) buffer_read(i);
    const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(C::COLS * h);
    float* slots = &s_sx[0][threadIdx.x - 128];
    uint8_t* out = smem + C::STAGES * C::STAGE_BYTES + (warp - 4) * C::OUT_BYTES;
    uint32_t res_phase = 0;
    int stage = 0;
    uint32_t phase = 0, buf = 0;
    bool ok = true;
    for (int u = group; u < a.units && ok; u += groups) {
      const int row0 = (u % a.m_tiles) * C::BM + 32 * q;
      const int col0 = (u / a.m_tiles) * C::BN + C::COLS * h;
      const bool live = row0 < a.M && col0 < a.N;  // warp-uniform
      if (a.residual && splits == 1 && lane == 0) {
        bulk_wait_group_read0();
        mbar_arrive_expect_tx(&res_bar[warp - 4], C::OUT_BYTES);
        tma_load_2d(out, &tmR, &res_bar[warp - 4], col0, row0);
      }
      // rows and columns past the output use the last ones' scales and are not stored
      const int n = kb1 - kb0;
      ScaleStream<32 * C::EPI_WARPS> scales;
      scales.start(a.sx + static_cast<int64_t>(kb0) * a.M + min(row0 + lane, a.M - 1),
                   a.sw + static_cast<int64_t>(min(col0, a.N - 1) >> 7) * a.blocks + kb0, n, slots, a.M, lane);
      float acc[C::COLS];
#pragma unroll
      for (int j = 0; j < C::COLS; ++j) acc[j] = 0.0f;
      float sc = scales.next(0, a.M, lane);
      bool ready = false;
      for (int b = 0; b < n; ++b) {
        if (!__all_sync(0xffffffffu, ready) && !warp_wait(&done_bar[stage], phase, a.budget, &s_abort, 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the next block's scale and barrier and the second load overlap the
        // first load and the products
        uint32_t p0[32], p1[32];
        tmem_ld_32x32b_x32(tbase + buf, p0);
        const float sc1 = b + 1 < n ? scales.next(b + 1, a.M, lane) : 0.0f;
        tmem_ld_wait();
        tmem_ld_32x32b_x32(tbase + buf + 32, p1);
        add_scaled32(acc, p0, sc);
        tmem_ld_wait();
        buffer_read(stage + C::BUFS < C::STAGES ? stage + C::BUFS : stage + C::BUFS - C::STAGES);
        buf = (buf + C::BN) & (C::BUFS * C::BN - 1);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        ready = mbar_test_wait(&done_bar[stage], phase);
        add_scaled32(acc + 32, p1, sc);
        sc = sc1;
      }
      if (!ok) break;
      if (splits > 1) {
        // the ring is idle: every block of this CTA's range has been consumed
        write_sums(smem_u32(smem), 32 * q + lane, acc, C::COLS * h / 4);
      } else {
        if (a.residual) {
          if (!warp_wait(&res_bar[warp - 4], res_phase, a.budget, &s_abort, 0)) break;
          res_phase ^= 1u;
        } else {
          if (lane == 0) bulk_wait_group_read0();
          __syncwarp();
        }
#pragma unroll
        for (int c = 0; c < C::COLS; c += 8) {
          const uint32_t at = smem_u32(out) + lane * 128 + (((c / 8) ^ (lane & 7)) << 4);
          if (a.residual) {
            const uint4 rv = ld_shared_v4(at);
            const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[c + 2 * j] += __uint_as_float(rw[j] << 16);
              acc[c + 2 * j + 1] += __uint_as_float(rw[j] & 0xFFFF0000u);
            }
          }
          st_shared_v4(at, bf16x2(acc[c], acc[c + 1]), bf16x2(acc[c + 2], acc[c + 3]), bf16x2(acc[c + 4], acc[c + 5]),
                       bf16x2(acc[c + 6], acc[c + 7]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && live) {
          tma_store_2d(&tmY, out, col0, row0);
          bulk_commit_group();
        }
      }
    }
    if (!ok && splits > 1)  // the permuted groups of a warp's columns stay in their half of the row
      give_up_sums(reinterpret_cast<float*>(smem) + (32 * q + lane) * C::BN + C::COLS * h, C::COLS, 1);
    if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before();
  __syncwarp();
  if (splits > 1) {
    cluster_sync();  // every CTA's sums are in its shared memory
    const int gave_up = s_abort;
    const int m0 = (group % a.m_tiles) * C::BM, n0 = (group / a.m_tiles) * C::BN;
    const int items = min(C::BM, a.M - m0) * (C::BN / 4);
    const uint32_t sums = smem_u32(smem);
    // four columns of Y per item, added in the order of the blocks
    for (int i = rank * C::THREADS + static_cast<int>(threadIdx.x); i < items; i += splits * C::THREADS) {
      const int j = i / (C::BN / 4), c = i % (C::BN / 4), n = n0 + 4 * c;
      if (n >= a.N) continue;  // N % 8 == 0: four columns are in or out as a whole
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int r = 0; r < splits; ++r) add4(y, read_sums(mapa_shared(sums, r), j, c));
      store4(a, y, m0 + j, n);
    }
    __syncwarp();
    cluster_sync_relaxed();  // no CTA leaves while another reads its sums
    if (gave_up) let_copies_land();
  } else {
    __syncthreads();
    if (s_abort) let_copies_land();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::BUFS * C::BN);
  }
}

// ---------------------------------------------------------------------------
// Decode: 128 weight rows (MMA rows, TMEM lanes) x NT tokens (columns), so the
// MMA and the epilogue are as narrow as the tokens (one tile of them) and the
// weights stream once.  Clusters, roles and barriers as in the kernel above,
// with four epilogue warps; the token scales of CHUNK blocks at a time go
// through shared memory, copied by the epilogue warps one chunk ahead.
//
// What bounds it: HBM for the weights, behind about 3 us of start, first round
// trip and cluster sum.  8 x 3584 x 18944 14.4 us (28 tiles of four CTAs, 4.7
// TB/s), 4 x 37888 x 3584 23.8 (296 tiles of one, 5.7), 1 x 4608 x 3584 6.4 (36
// tiles of three).  Widths of 75 to 147 tiles do not fill the chip: tiles are
// split only while all clusters are resident at once, so 1 x 10240 x 3584 runs
// 80 CTAs and takes 11.3 us (3.3 TB/s).
template <int NT>
struct ColsTile {
  static constexpr int BN = 128;  // weight rows
  static constexpr int X_BYTES = NT * kRowBytes;
  static constexpr int STAGE_BYTES = kTileBytes + X_BYTES;
  static constexpr int STAGES = (192 * 1024) / STAGE_BYTES > 10 ? 10 : (192 * 1024) / STAGE_BYTES;
  static constexpr int BUFS = 4;  // accumulator buffers
  static constexpr int CHUNK = 8;  // blocks of scales per copy
  static constexpr int EPI_WARPS = 4;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int TMEM_COLS = BUFS * NT;  // a power of two, >= 32
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024;
  // kind::f8f6f4, E4M3 x E4M3, fp32 accumulator, N = NT, M = 128
  static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(NT >> 3) << 17) | (uint32_t(BN >> 4) << 24);
  static_assert(NT * BN * 4 <= STAGES * STAGE_BYTES, "the cluster's sums fit the operand ring");
  static_assert(BUFS <= STAGES, "a stage's barrier is armed after its buffer's previous block");
  static_assert(TMEM_COLS <= kTmemColumns, "TMEM budget");
};

template <int NT>
__global__ void __launch_bounds__(ColsTile<NT>::THREADS, 1)
gemm_block_cols_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const BlockArgs a, const int splits) {
  using C = ColsTile<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];  // operands of a block, buffer read
  __shared__ __align__(8) uint64_t done_bar[C::STAGES];  // block accumulated
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ __align__(16) float s_sx[2][C::CHUNK][NT];  // token scales of two chunks of blocks
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int group = static_cast<int>(blockIdx.x) / splits;
  const int groups = static_cast<int>(gridDim.x) / splits;
  // blocks <= 2^24, splits <= 8
  const int kb0 = static_cast<int>(static_cast<uint32_t>(a.blocks * rank) / static_cast<uint32_t>(splits));
  const int kb1 = static_cast<int>(static_cast<uint32_t>(a.blocks * (rank + 1)) / static_cast<uint32_t>(splits));

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full_bar[i], 1 + C::EPI_WARPS);
      mbar_init(&done_bar[i], 1);
    }
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  const int first = group * C::BN;  // weight row of the first tile
  keep(kb0, kb1, first);            // computed before the wait
  // the first weights come into L2 while the previous kernel ends (1 x 4608 x
  // 3584: 6.7 -> 6.2 us back to back; all of the ring's stages: 7.1 us)
  if (warp == 0 && elect_one())
    for (int b = kb0; b < min(kb1, kb0 + kPrefetchBlocks); ++b) tma_prefetch_2d(&tmW, b * kRowBytes, first);
  griddep_wait();
  griddep_launch_dependents();

  if ((warp == 0 || warp == 2) && elect_one()) {
    // ----------------------------------------------------- producers: w, x
    const bool is_w = warp == 0;
    const CUtensorMap* map = is_w ? &tmW : &tmX;
    uint8_t* dst = smem + (is_w ? 0 : kTileBytes);
    int it = 0, stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = group; u < a.units && ok; u += groups) {
      const int row0 = is_w ? first + (u - group) * C::BN : 0;
      for (int b = kb0; b < kb1; ++b, ++it) {
        if (it >= C::STAGES && !bounded_wait(&done_bar[stage], phase ^ 1u, a.budget, &s_abort, 0)) {
          ok = false;
          break;
        }
        if (is_w) mbar_arrive_expect_tx(&full_bar[stage], C::STAGE_BYTES);
        tma_load_2d(dst + stage * C::STAGE_BYTES, map, &full_bar[stage], b * kRowBytes, row0);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1 && elect_one()) {
    // ----------------------------------------------------------- MMA issuer
    const uint64_t wd = sdesc_kmajor_sw128(smem_u32(smem)), xd = sdesc_kmajor_sw128(smem_u32(smem) + kTileBytes);
    int stage = 0;
    uint32_t phase = 0, buf = 0;
    bool ok = true;
    for (int u = group; u < a.units && ok; u += groups) {
      for (int b = kb0; b < kb1; ++b) {
        if (!bounded_wait(&full_bar[stage], phase, a.budget, &s_abort, 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(stage) * (C::STAGE_BYTES >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f8f6f4(tmem + buf, wd + off + 2 * j, xd + off + 2 * j, C::IDESC, j > 0);
        umma_commit(&done_bar[stage]);
        buf = (buf + NT) & (C::TMEM_COLS - 1);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    umma_commit(&drain_bar);
    const long long t0 = clock64();
    while (!mbar_try_wait(&drain_bar, 0) && clock64() - t0 < 4 * a.budget + 1000000) {
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    constexpr int CH = NT < 32 ? NT : 32;  // columns per TMEM load
    const int q = warp & 3;
    const int t = static_cast<int>(threadIdx.x) - 128;
    auto buffer_read = [&](int stage) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(&full_bar[stage]);
    };
#pragma unroll
    for (int i = 0; i < C::BUFS; ++i) buffer_read(i);
    const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * q) << 16);
    int stage = 0;
    uint32_t phase = 0, buf = 0;
    bool ok = true;
    for (int u = group; u < a.units; u += groups) {
      const int n0 = u * C::BN;
      const float* swp = a.sw + static_cast<int64_t>(u) * a.blocks;
      // columns past the last token use its scales and are not stored
      auto copy_chunk = [&](int b, int half) {
        for (int i = t; i < C::CHUNK * NT; i += 32 * C::EPI_WARPS)
          if (b + i / NT < kb1)
            cp_async4(smem_u32(&s_sx[half][0][i]), a.sx + static_cast<int64_t>(b + i / NT) * a.M + min(i % NT, a.M - 1));
        cp_async_commit();
      };
      copy_chunk(kb0, 0);
      float w8 = 0.0f, w8n = __ldg(swp + min(kb0 + lane, a.blocks - 1));  // weight scales, one per lane
      float acc[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = 0.0f;
      int half = 0;
      for (int b0 = kb0; b0 < kb1; b0 += C::CHUNK) {
        w8 = w8n;
        w8n = __ldg(swp + min(b0 + C::CHUNK + lane, a.blocks - 1));
        cp_async_wait<0>();
        // every warp's part of this chunk has landed, and the other chunk's
        // buffer has been read by all
        epilogue_sync(32 * C::EPI_WARPS);
        copy_chunk(b0 + C::CHUNK, half ^ 1);
        const int b1 = min(b0 + C::CHUNK, kb1);
        for (int b = b0; b < b1 && ok; ++b) {
          const float w = __shfl_sync(0xffffffffu, w8, b - b0);
          if (!warp_wait(&done_bar[stage], phase, a.budget, &s_abort, 0)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float4* sc = reinterpret_cast<const float4*>(&s_sx[half][b - b0][0]);
#pragma unroll
          for (int c = 0; c < NT; c += CH) {
            uint32_t p[CH];
            if constexpr (CH == 32)
              tmem_ld_32x32b_x32(tbase + buf + c, p);
            else
              tmem_ld_32x32b_x16(tbase + buf + c, p);
            tmem_ld_wait();
            if (c + CH == NT) buffer_read(stage + C::BUFS < C::STAGES ? stage + C::BUFS : stage + C::BUFS - C::STAGES);
#pragma unroll
            for (int j = 0; j < CH; j += 4) {
              const float4 s4 = sc[(c + j) / 4];
              acc[c + j] = fmaf(__uint_as_float(p[j]), s4.x * w, acc[c + j]);
              acc[c + j + 1] = fmaf(__uint_as_float(p[j + 1]), s4.y * w, acc[c + j + 1]);
              acc[c + j + 2] = fmaf(__uint_as_float(p[j + 2]), s4.z * w, acc[c + j + 2]);
              acc[c + j + 3] = fmaf(__uint_as_float(p[j + 3]), s4.w * w, acc[c + j + 3]);
            }
          }
          buf = (buf + NT) & (C::TMEM_COLS - 1);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        half ^= 1;
      }
      cp_async_wait<0>();
      epilogue_sync(32 * C::EPI_WARPS);  // the next tile's first chunk overwrites this tile's last
      const int n = n0 + 32 * q + lane;
      if (!ok) continue;
      if (splits > 1) {
        // the ring is idle: every block has been consumed
        float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[j * C::BN + 32 * q + lane] = acc[j];
      } else if (n < a.N) {
        if (a.residual) {
          // all of them on the way before the first is used (rows past the
          // last token read the last one's): one at a time, 37 x 96 x 352 took
          // 11.2 us
          __nv_bfloat16 r[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) r[j] = a.residual[static_cast<size_t>(min(j, a.M - 1)) * a.N + n];
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[j] += __bfloat162float(r[j]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j < a.M) a.Y[static_cast<size_t>(j) * a.N + n] = __float2bfloat16_rn(acc[j]);
      }
    }
    if (!ok && splits > 1) give_up_sums(reinterpret_cast<float*>(smem) + 32 * q + lane, NT, C::BN);
  }

  tc_fence_before();
  __syncwarp();
  if (splits > 1) {
    cluster_sync();  // every CTA's sums are in its shared memory
    const int gave_up = s_abort;
    const int n0 = group * C::BN;
    const int items = a.M * (C::BN / 4);
    const uint32_t sums = smem_u32(smem);
    // four columns of Y per item, added in the order of the blocks
    for (int i = rank * C::THREADS + static_cast<int>(threadIdx.x); i < items; i += splits * C::THREADS) {
      const int j = i / (C::BN / 4), n = n0 + 4 * (i % (C::BN / 4));
      if (n >= a.N) continue;  // N % 8 == 0: four columns are in or out as a whole
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int r = 0; r < splits; ++r)
        add4(y, ld_shared_cluster_f4(mapa_shared(sums + static_cast<uint32_t>(i) * 16u, r)));
      store4(a, y, j, n);
    }
    __syncwarp();
    cluster_sync_relaxed();  // no CTA leaves while another reads its sums
    if (gave_up) let_copies_land();
  } else {
    __syncthreads();
    if (s_abort) let_copies_land();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// -------------------------------------------------------------- host side --
constexpr int kMaxSplits = 8;  // portable cluster size

BlockArgs make_block_args(const BlockLinear& l, int bm, int bn) {
  BlockArgs a;
  a.sx = l.s_x;
  a.sw = l.s_w;
  a.residual = static_cast<const __nv_bfloat16*>(l.residual);
  a.Y = static_cast<__nv_bfloat16*>(l.Y);
  a.M = static_cast<int>(l.M);
  a.N = static_cast<int>(l.N);
  a.blocks = static_cast<int>((l.K + 127) / 128);
  a.m_tiles = static_cast<int>((l.M + bm - 1) / bm);
  a.n_tiles = static_cast<int>((l.N + bn - 1) / bn);
  a.units = a.m_tiles * a.n_tiles;
  a.budget = l.starve ? kStarvedBudgetCycles : kWaitBudgetCycles;
  return a;
}

// l.starve: boxes of half the token rows, so that no stage ever has all its
// bytes and every wait for one runs out (the failure self test).
bool make_block_maps(const BlockLinear& l, uint32_t x_rows, CUtensorMap* tx, CUtensorMap* tw) {
  const uint64_t k = static_cast<uint64_t>(l.K);
  return make_map(tx, l.xq, k, static_cast<uint64_t>(l.M), k, l.starve ? x_rows / 2 : x_rows) &&
         make_map(tw, l.wq, k, static_cast<uint64_t>(l.N), k, 128);
}

// Clusters of `size` CTAs of a kernel that the current device holds at once
// (cached per device; 0 when the query fails).
template <typename K>
int clusters_resident(K kern, int size, int threads, int smem, std::atomic<int> (&cache)[kMaxDevices]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return 0;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(size));
  cfg.blockDim = dim3(static_cast<unsigned int>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned int>(size);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 0) {
    cudaGetLastError();
    n = 0;
  }
  cache[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

int pair_clusters(bool split) {
  static std::atomic<int> cache[2][kMaxDevices];
  auto kern = split ? gemm_block_pair_kernel<true> : gemm_block_pair_kernel<false>;
  const int n = clusters_resident(kern, split ? 4 : 2, PairTile::THREADS, PairTile::SMEM_BYTES, cache[split]);
  return n > 0 ? n : 1;
}

int rows_clusters(int splits) {
  using C = RowsTile;
  static std::atomic<int> cache[kMaxSplits + 1][kMaxDevices];
  return clusters_resident(gemm_block_rows_kernel, splits, C::THREADS, C::SMEM_BYTES, cache[splits]);
}

template <int NT>
int cols_clusters(int splits) {
  using C = ColsTile<NT>;
  static std::atomic<int> cache[kMaxSplits + 1][kMaxDevices];
  return clusters_resident(gemm_block_cols_kernel<NT>, splits, C::THREADS, C::SMEM_BYTES, cache[splits]);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Time of a tile split over a cluster that does not depend on its depth (start,
// first round trip, sum), in ns, and of a block of K: clusters of four start
// fastest (333 x 1000 x 1040, by 1, 2, 3, 4 CTAs: 7.1, 7.6, 7.0, 6.7 us; 300 x 512
// x 3584, by 4, 5, 6, 7, 8: 7.5, 7.9, 7.9, 7.7, 7.7).  Fitted to tiles of 128
// tokens.  The columns kernel, whose blocks take less, chooses by the same
// figures: over 60 shapes of 1 to 64 tokens the plan took 2.4% longer than the
// best on average.
constexpr int64_t kBlockNs = 338;
int64_t split_ns(int64_t blocks, int splits) {
  return (splits < 4 ? 5850 : splits == 4 ? 5600 : 6500) + kBlockNs * ceil_div(blocks, splits);
}

// CTAs that share a tile: the fastest size that keeps every cluster resident at
// once, with at least two blocks of K for each CTA; 1 where none does.
template <typename Resident>
int choose_splits(int64_t tiles, int64_t blocks, Resident resident) {
  int best = 1;
  for (int splits = 2; splits <= kMaxSplits && blocks >= 2 * splits; ++splits)
    if (tiles <= resident(splits) && (best == 1 || split_ns(blocks, splits) < split_ns(blocks, best))) best = splits;
  return best;
}

// Tiles of one CTA each (grid capped at the SMs, which loop), or of a cluster.
template <typename Kernel, typename... Args>
cudaError_t launch_tiles(Kernel kern, int threads, int smem, int units, int splits, cudaStream_t s, Args... args) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count();
  if (splits == 1)
    return launch_pdl(kern, dim3(static_cast<unsigned int>(units < sms ? units : sms)), dim3(threads), smem, s,
                      args..., 1);
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned int>(units * splits)), dim3(threads), splits, smem, s,
                            args..., splits);
}

cudaError_t run_block_pair(const BlockLinear& l, bool split, cudaStream_t s) {
  using C = PairTile;
  CUtensorMap tx, tw, ty, tr;
  const uint64_t cols = static_cast<uint64_t>(l.N), rows = static_cast<uint64_t>(l.M);
  if (!make_block_maps(l, 128, &tx, &tw) || !make_out_map(&ty, l.Y, cols, rows)) return cudaErrorInvalidValue;
  tr = ty;  // not read without a residual
  if (l.residual && !make_out_map(&tr, const_cast<void*>(l.residual), cols, rows)) return cudaErrorInvalidValue;
  const BlockArgs a = make_block_args(l, C::BM, C::BN);
  auto kern = split ? gemm_block_pair_kernel<true> : gemm_block_pair_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int resident = pair_clusters(false);
  const int clusters = split || a.units < resident ? a.units : resident;
  const int ctas = split ? 4 : 2;
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned int>(ctas * clusters)), dim3(C::THREADS), ctas,
                            C::SMEM_BYTES, s, tx, tw, ty, tr, a);
}

cudaError_t run_block_rows(const BlockLinear& l, int splits, cudaStream_t s) {
  using C = RowsTile;
  CUtensorMap tx, tw, ty, tr;
  const uint64_t cols = static_cast<uint64_t>(l.N), rows = static_cast<uint64_t>(l.M);
  if (!make_block_maps(l, C::BM, &tx, &tw) || !make_out_map(&ty, l.Y, cols, rows)) return cudaErrorInvalidValue;
  tr = ty;  // not read without a residual
  if (l.residual && !make_out_map(&tr, const_cast<void*>(l.residual), cols, rows)) return cudaErrorInvalidValue;
  const BlockArgs a = make_block_args(l, C::BM, C::BN);
  return launch_tiles(gemm_block_rows_kernel, C::THREADS, C::SMEM_BYTES, a.units, splits, s, tx, tw, ty, tr, a);
}

template <int NT>
cudaError_t run_block_cols(const BlockLinear& l, int splits, cudaStream_t s) {
  using C = ColsTile<NT>;
  CUtensorMap tx, tw;
  if (!make_block_maps(l, NT, &tx, &tw)) return cudaErrorInvalidValue;
  const BlockArgs a = make_block_args(l, NT, C::BN);
  return launch_tiles(gemm_block_cols_kernel<NT>, C::THREADS, C::SMEM_BYTES, a.units, splits, s, tx, tw, a);
}

}  // namespace

// Up to 64 tokens: columns of 16, 32 or 64 tokens (in columns twice as wide 1 x
// 4608 x 3584 takes 6.9 us instead of 6.2, 32 x 3584 x 18944 19.4 instead of 15.4).
// Past 32, the tiles of 128 tokens start 0.7 us later but take less time for a
// block, which pays from about 20 blocks in a row on (columns / rows, us: 33 x
// 3584 x 3584, 7 blocks, 7.7 / 8.4; 48 x 18944 x 2048, 16, 12.0 / 12.1; 64 x 3584 x
// 18944, 37, 19.7 / 18.0; 64 x 37888 x 3584, 56, 31.1 / 26.7), and, which the rule
// does not know, for one or two blocks (64 x 5624 x 160: 5.3 / 4.0).
//
// More than 64 tokens: the plan with the least estimated time, in ns of a cold
// call: a start, and for every wave of tiles the blocks of K in turn.
// (pair / pair, K in two / tiles of 128, us: 512 x 3584 x 3584 16.5 / 14.8 /
// 12.4; 1024 x 3584 x 3584 17.4 / 28.9 / 21.5; 512 x 3584 x 18944 64 / 41 / 52;
// 256 x 3584 x 18944 67 / 41 / 29; 1024 x 3584 x 18944 69 / 93 / 104.)  Every plan
// measured on 110 other shapes of 65 to 4580 tokens, widths to 37888 and depths
// to 18944, than the constants were fitted to: the one chosen took 0.3% longer
// than the best on average, 8% at most (up to 64 tokens, 60 shapes, 2.4% and 32%,
// the most at 64 x 5624 x 160).
BlockPlan plan_linear_fp8_block(int64_t M, int64_t N, int64_t K) {
  const int64_t blocks = ceil_div(K, 128);
  const int64_t columns = ceil_div(N, 128), tiles = ceil_div(M, 128) * columns;
  if (M <= 16) return {kBlockCols, choose_splits(columns, blocks, cols_clusters<16>)};
  if (M <= 32) return {kBlockCols, choose_splits(columns, blocks, cols_clusters<32>)};
  int splits = choose_splits(tiles, blocks, rows_clusters);
  if (M <= 64) {
    const int64_t in_a_row = ceil_div(tiles, splits > 1 ? tiles : device_sm_count()) * ceil_div(blocks, splits);
    if (in_a_row <= 20) return {kBlockCols, choose_splits(columns, blocks, cols_clusters<64>)};
    return {kBlockRows, splits};
  }
  const int64_t units = ceil_div(M, 256) * ceil_div(N, 256);
  const int64_t pair = 2700 + ceil_div(units, pair_clusters(false)) * (1800 + 455 * blocks);
  const int64_t halves = ceil_div(units, pair_clusters(true)) * (8600 + 245 * blocks) - 1500;
  int64_t rows = 2600 + ceil_div(tiles, device_sm_count()) * (1000 + kBlockNs * blocks);
  if (splits > 1 && split_ns(blocks, splits) < rows)
    rows = split_ns(blocks, splits);
  else
    splits = 1;
  if (rows <= pair && rows <= halves) return {kBlockRows, splits};
  return {kBlockPair, blocks > 1 && halves < pair ? 4 : 2};
}

bool block_plan_valid(const BlockPlan& plan, int64_t M, int64_t K) {
  const int64_t blocks = ceil_div(K, 128);
  if (plan.kernel == kBlockPair) return plan.ctas == 2 || (plan.ctas == 4 && blocks >= 2);
  if (plan.kernel != kBlockRows && (plan.kernel != kBlockCols || M > 64)) return false;
  return plan.ctas >= 1 && plan.ctas <= kMaxSplits && plan.ctas <= blocks;
}

cudaError_t launch_linear_fp8_block(const BlockLinear& l, const BlockPlan& plan, cudaStream_t s) {
  if (plan.kernel == kBlockPair) return run_block_pair(l, plan.ctas == 4, s);
  if (plan.kernel == kBlockRows) return run_block_rows(l, plan.ctas, s);
  if (l.M <= 16) return run_block_cols<16>(l, plan.ctas, s);
  if (l.M <= 32) return run_block_cols<32>(l, plan.ctas, s);
  return run_block_cols<64>(l, plan.ctas, s);
}

cudaError_t block_linear_status_word(unsigned int** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), g_vlaq_block_status);
}

}  // namespace vlaq
