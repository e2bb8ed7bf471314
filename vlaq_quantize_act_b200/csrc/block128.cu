// FP8 quantizers with one scale per block of 128, and the residual update
// between two blocks of a decoder (post norm, gate, residual scale, add, pre
// norm) with a bf16 or FP8 block output.
//
//   s = max |v| / 448 over a block (1 x 128 of a token row, 128 x 128 of a
//   weight), code = E4M3_rne_sat(v / s), 0 where s = 0; the arithmetic of the
//   per-row FP8 quantizer in smaller scopes.
//
// Layouts, each chosen so that a thread's loads are in flight together and a
// block's amax needs few exchanges:
//   quant_blocks_kernel          4 lanes per 1 x 128 block, 32 elements each
//   quant_rotated_spread_kernel  16 lanes per block, 8 elements each (few blocks)
//   quant_rotated_kernel         one 64-element rotation per thread, tiles by TMA
//   quant_weight_block_kernel    a CTA per 128 x 128 block, 64 elements a thread
//   norm_rows_kernel             a CTA per row, 16-element chunks
// For one row all are bound by the launch and one memory round trip.  For many
// rows (2 or 4 bytes in, 1 to 4 out per element) the weight blocks and the bf16
// residual norm are bound by HBM (5.8 to 6.4 TB/s; plain activation blocks 5.1 to
// 5.3), the rotations by their instructions as well (5.1); rows with a norm and an
// FP8 result by the chain of steps of a row, of which a CTA has one at a time:
// 4580 x 3584 RMSNorm to FP8 18.2 us (2.7 TB/s), rotated 20.8, residual norm to
// FP8 27.8 (4.1), rotated and gated 32.7.
//
// Times are device times of a call, in a CUDA graph of calls over buffers larger
// than L2, where nothing else is said; a pair of times with an arrow is one
// change, measured before and after it.
//
// Sums of squares use a fixed tree of 256 lanes, so a row's result does not
// depend on how many rows the call has or on the CTA's thread count: lane l
// owns the 16-element chunks l, l + 256, ... and adds them in element order
// with fused multiply-adds; an XOR butterfly 16, 8, 4, 2, 1 joins each group of
// 32 lanes and a butterfly 1, 2, 4 the eight groups.  A thread of a CTA with T
// < 256 threads carries 256 / T of these lanes.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"
#include "tensor_map.h"

namespace vlaq {

__device__ unsigned int g_vlaq_block128_status = 0;

namespace {

constexpr int kTreeLanes = 256;

__device__ __forceinline__ uint4 pack_bf16x8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// max |v| of 8 bf16 values, kept packed (the max of bf16 values is one of them).
__device__ __forceinline__ float absmax_bf16x8(const uint4& a) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  __nv_bfloat162 h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t aw = w[j] & 0x7FFF7FFFu;  // |x| of both halves
    h[j] = *reinterpret_cast<const __nv_bfloat162*>(&aw);
  }
  const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ float absmax8(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  return m;
}

// Normalised WHT of the 64-block on lanes 8 g .. 8 g + 7, 8 values each:
// stages h = 1, 2, 4 in the lane, 8, 16, 32 across lanes (xor 1, 2, 4), then
// x 1/8 (exact): the stages of the sequential butterfly in its order, each
// sum or difference rounded once.  Executed by the whole warp.
__device__ __forceinline__ void wht64_chunk(float* v, int lane) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = __fadd_rn(a, b);
        v[i + h] = __fsub_rn(a, b);
      }
    }
  }
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) {
    const float sg = (lane & x) != 0 ? -1.0f : 1.0f;  // upper lane: partner - own
    const float2 s2 = make_float2(sg, sg);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 p = make_float2(__shfl_xor_sync(0xffffffffu, v[i], x), __shfl_xor_sync(0xffffffffu, v[i + 1], x));
      const float2 r = __ffma2_rn(make_float2(v[i], v[i + 1]), s2, p);
      v[i] = r.x;
      v[i + 1] = r.y;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], 0.125f);
}

// Scale of the 1 x 128 block on 16 adjacent lanes.  Executed by the warp.
__device__ __forceinline__ float block_scale16(const float* v) {
  float m = absmax8(v);
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  return row_global<1>(m);
}

// Largest of all threads' values (>= 0).  Executed by the whole CTA.
__device__ __forceinline__ float block_amax(float m, float* s_max) {
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // bit order is value order
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) m = fmaxf(m, s_max[w]);
  return m;
}

// ------------------------------------------------------ activation blocks --
// Without a norm the blocks of all rows are independent.
struct BlocksArgs {
  const __nv_bfloat16* X;
  int64_t rows, K;
  int64_t blocks;                  // per row
  int64_t total;                   // rows * blocks
  unsigned long long inv_blocks;   // floor(2^64 / blocks) + 1 (blocks > 1)
  uint8_t* codes;
  float* scales;                   // [blocks][rows]
};

// Row of block i: exact while i * blocks < 2^64.
__device__ __forceinline__ int64_t block_row(const BlocksArgs& a, int64_t i) {
  return a.blocks == 1 ? i : static_cast<int64_t>(__umul64hi(i, a.inv_blocks));
}

constexpr int kBlocksThreads = 256;
constexpr int kPlainBlocks = kBlocksThreads / 4;

// Four lanes per block, chunks sub, sub + 4, sub + 8, sub + 12 of it each: the
// four loads are in flight together, every load and store of the four lanes
// covers whole sectors, and the amax takes two shuffles and the scale and its
// reciprocal are formed once per 32 elements of a thread.
__global__ void __launch_bounds__(kBlocksThreads) quant_blocks_kernel(const BlocksArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 3;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kPlainBlocks + (threadIdx.x >> 2);
  const int64_t row = block_row(a, i), b = i - row * a.blocks;
  const int left = i < a.total ? static_cast<int>(min(static_cast<int64_t>(128), a.K - b * 128)) - 8 * sub : 0;
  const int64_t off = row * a.K + b * 128 + 8 * sub;
  uint4 d[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    d[u] = 32 * u < left ? __ldg(reinterpret_cast<const uint4*>(a.X + off + 32 * u)) : make_uint4(0, 0, 0, 0);
  float m = fmaxf(fmaxf(absmax_bf16x8(d[0]), absmax_bf16x8(d[1])), fmaxf(absmax_bf16x8(d[2]), absmax_bf16x8(d[3])));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float s = row_global<1>(m);
  const Divisor dv = make_divisor(s);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float v[8];
    unpack_bf16x8(d[u], v);
    const uint2 w = e4m3_codes8(v, dv);
    if (32 * u < left) *reinterpret_cast<uint2*>(a.codes + off + 32 * u) = w;
  }
  if (sub == 0 && i < a.total) a.scales[b * a.rows + row] = s;
}

// Rotated, few blocks: 16 lanes per block, the rotation over 8 of them.
constexpr int kSpreadBlocks = kBlocksThreads / 16;

__global__ void __launch_bounds__(kBlocksThreads) quant_rotated_spread_kernel(const BlocksArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 15;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kSpreadBlocks + (threadIdx.x >> 4);
  const int64_t row = block_row(a, i), b = i - row * a.blocks;
  const int64_t k = b * 128 + 8 * sub;
  const bool in = i < a.total && k < a.K;
  float v[8];
  unpack_bf16x8(in ? __ldg(reinterpret_cast<const uint4*>(a.X + row * a.K + k)) : make_uint4(0, 0, 0, 0), v);
  wht64_chunk(v, threadIdx.x & 31);
  const float s = block_scale16(v);
  const uint2 w = e4m3_codes8(v, make_divisor(s));
  if (in) {
    *reinterpret_cast<uint2*>(a.codes + row * a.K + k) = w;
    if (sub == 0) a.scales[b * a.rows + row] = s;
  }
}

// ------------------------------------------------------------ weight blocks --
// One CTA per 128 x 128 block: 16 lanes cover a row's 128 columns, 16 rows at
// a time; the whole block stays in registers (8 chunks of bf16 per thread)
// between the amax and the codes, so W is read once.  HBM-bound: 37888 x 3584
// in 63.5 us, 6.42 TB/s (64 registers, four CTAs per SM; with the 104 of an
// unbounded build, two CTAs, 85 us; with 40, spilled, 96 us).
constexpr int kWeightThreads = 256;

__global__ void __launch_bounds__(kWeightThreads, 4)
    quant_weight_block_kernel(const __nv_bfloat16* W, int64_t N, int64_t K, uint8_t* codes, float* scales) {
  __shared__ float s_max[kWeightThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const uint32_t k_blocks = static_cast<uint32_t>((K + 127) / 128);
  const int64_t nb = blockIdx.x / k_blocks, kb = blockIdx.x % k_blocks;
  const int64_t k = kb * 128 + 8 * sub;
  const int64_t first = (nb * 128 + r0) * K + k;  // this thread's first chunk, 16 rows to the next
  const int rows = static_cast<int>(min(static_cast<int64_t>(128), N - nb * 128));
  uint4 d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    d[i] = r0 + 16 * i < rows && k < K ? __ldg(reinterpret_cast<const uint4*>(W + first + 16 * i * K))
                                       : make_uint4(0, 0, 0, 0);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, absmax_bf16x8(d[i]));
  m = block_amax(m, s_max);
  const float s = row_global<1>(m);
  const Divisor dv = make_divisor(s);
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float t[8];
    unpack_bf16x8(d[i], t);
    const uint2 w = e4m3_codes8(t, dv);
    if (r0 + 16 * i < rows && k < K) *reinterpret_cast<uint2*>(codes + first + 16 * i * K) = w;
  }
}

// ------------------------------------------------- rotated blocks, many rows --
// Rotations of plain bf16 input (weights, activations without a norm): a
// thread transforms one whole 64-element block in its registers, so nothing
// is exchanged between lanes.  A CTA takes 128 rows x 128 columns at a time,
// as two TMA boxes of 128 rows x 64 columns (128-byte swizzle), one tile
// ahead; thread t has row t % 128 of box t / 128, so a quarter warp's 16-byte
// reads fall on eight different swizzled positions; the codes leave by one
// TMA store per tile (stored by the threads, 64 bytes of a row each, 37888 x
// 3584 took 95 us).  37888 x 3584: 80 us, 5.1 TB/s; 1024 x 18944: 14.7 us.  Two
// CTAs per SM (the 64 values of a thread) alternate between memory and the
// about 500 instructions of 64 elements, of which the rotation has 220.
constexpr int kRotThreads = 256;
constexpr int kRotBoxBytes = 128 * 128;
constexpr int kRotSmem = (2 * 2 + 1) * kRotBoxBytes + 1024;

// Unnormalised WHT of 64 values (8 times the normalised one), stages in the
// sequential order, each sum and difference rounded once; the packed stages
// as in wht64_lanes.
__device__ __forceinline__ void wht64_thread(float2 (&v)[32]) {
  const float2 m1 = make_float2(-1.0f, -1.0f);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = make_float2(__fadd_rn(v[i].x, v[i].y), __fsub_rn(v[i].x, v[i].y));
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if ((i & h) == 0) {
        const float2 a = v[i], b = v[i + h];
        v[i] = __fadd2_rn(a, b);
        v[i + h] = __ffma2_rn(b, m1, a);
      }
    }
  }
}

struct RotArgs {
  int64_t rows;
  uint32_t k_blocks, tiles;
  float* scales;
  long long budget;
};

template <bool WEIGHT>
__global__ void __launch_bounds__(kRotThreads, 2)
    quant_rotated_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap out_map,
                         const RotArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[2];
  __shared__ float s_max[kRotThreads / 32];
  __shared__ float s_half[kRotThreads];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (threadIdx.x == 0) {
    prefetch_tensormap(&map);
    prefetch_tensormap(&out_map);
    mbar_init(&full_bar[0], 1);
    mbar_init(&full_bar[1], 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  auto load = [&](uint32_t tile, int buf) {
    if (threadIdx.x == 0 && tile < a.tiles) {
      const int row = static_cast<int>(tile / a.k_blocks * 128), col = static_cast<int>(tile % a.k_blocks * 128);
      mbar_arrive_expect_tx(&full_bar[buf], 2 * kRotBoxBytes);
      tma_load_2d(smem + 2 * buf * kRotBoxBytes, &map, &full_bar[buf], col, row);
      tma_load_2d(smem + (2 * buf + 1) * kRotBoxBytes, &map, &full_bar[buf], col + 64, row);
    }
  };
  uint8_t* out = smem + 4 * kRotBoxBytes;  // codes of the tile, 128-byte swizzle
  const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
  load(blockIdx.x, 0);
  int buf = 0;
  uint32_t phase = 0;
  for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    load(tile + gridDim.x, buf ^ 1);  // its previous contents were read before the last barrier
    // the whole CTA gives up or nobody, after its loads had the time to land
    if (!__syncthreads_and(mbar_wait(&full_bar[buf], phase, a.budget))) {
      if (threadIdx.x == 0) atomicOr(&g_vlaq_block128_status, kStatusTimeout);
      const long long t0 = clock64();
      while (clock64() - t0 < (1ll << 21)) {
      }
      break;
    }
    const uint32_t at = smem_u32(smem) + (2 * buf + half) * kRotBoxBytes + r * 128;
    float2 v[32];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 q = ld_shared_v4(at + ((c ^ (r & 7)) << 4));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[4 * c + j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    }
    wht64_thread(v);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = fmaxf(m, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
    // the transform's factor 1/8, exact here (sums of bf16 values are
    // multiples of 2^-133), goes into the amax and the divisor
    m = __fmul_rn(m, 0.125f);
    if (threadIdx.x == 0) bulk_wait_group_read0();  // the last tile's codes have left their buffer
    if (WEIGHT) {
      m = block_amax(m, s_max);
    } else {
      s_half[threadIdx.x] = m;
      __syncthreads();
      m = fmaxf(m, s_half[threadIdx.x ^ 128]);
    }
    const float s = row_global<1>(m);
    const Divisor dv = make_divisor(__fmul_rn(s, 8.0f));
    const uint32_t nb = tile / a.k_blocks, kb = tile - nb * a.k_blocks;
    const int64_t row = static_cast<int64_t>(nb) * 128 + r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2* p = v + 8 * i;
      const float t[16] = {p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y,
                           p[4].x, p[4].y, p[5].x, p[5].y, p[6].x, p[6].y, p[7].x, p[7].y};
      const uint2 lo = e4m3_codes8(t, dv), hi = e4m3_codes8(t + 8, dv);
      st_shared_v4(smem_u32(out) + r * 128 + (((4 * half + i) ^ (r & 7)) << 4), lo.x, lo.y, hi.x, hi.y);
    }
    if (WEIGHT) {
      if (threadIdx.x == 0) a.scales[tile] = s;
    } else if (half == 0 && row < a.rows) {
      a.scales[static_cast<int64_t>(kb) * a.rows + row] = s;
    }
    fence_proxy_async_smem();
    __syncthreads();  // the codes are written; the buffer, s_max and s_half have been read
    if (threadIdx.x == 0) {
      tma_store_2d(&out_map, out, static_cast<int>(kb * 128), static_cast<int>(nb * 128));  // clipped
      bulk_commit_group();
    }
    if (buf) phase ^= 1u;
    buf ^= 1;
  }
  if (threadIdx.x == 0) bulk_wait_group0();
}

// --------------------------------------------------- rows with a norm --
// One CTA per row, the row in registers (CPT chunks of 16 per thread).
//   RESID:  t = RMSNorm(y) (or y), t *= gate, c = h + alpha t, h' = bf16(c)
//   else:   c = x
//   then    v = RMSNorm(c) from the unrounded fp32 c (skipped when the call
//           asks for no x), and v as bf16, or rotated and as FP8 blocks.
enum { kOutBf16 = 0, kOutFp8 = 1 };

struct NormArgs {
  const __nv_bfloat16* h;  // residual stream, or x without RESID
  const __nv_bfloat16* y;
  const __nv_bfloat16* gamma_post;  // may be null: no post norm
  const __nv_bfloat16* gate;        // may be null: 1
  int64_t gate_rows;
  float alpha;
  const __nv_bfloat16* gamma_pre;
  float eps;
  __nv_bfloat16* h_out;
  __nv_bfloat16* x_out;  // kOutBf16; null: no x
  uint8_t* codes;        // kOutFp8
  float* scales;         // [blocks][rows]
  int64_t rows;
  int K;
  bool wide;  // every bf16 buffer is 32-byte aligned
};

// 16 bf16 values (32 bytes), in one access where their buffer's alignment
// allows it.  Plain, ordered accesses: outputs may overwrite inputs in place.
__device__ __forceinline__ void load_chunk(const __nv_bfloat16* p, bool wide, uint4& a, uint4& b) {
  if (wide) {
    ld_global_v8(p, a, b);
  } else {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
}

__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, bool wide, const float* v) {
  const uint4 a = pack_bf16x8(v), b = pack_bf16x8(v + 8);
  if (wide) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    st_global_v8(p, w);
  } else {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
}

// Sum of squares of a row in the 256-lane tree.  v: the thread's chunks in
// order (chunk i is chunk t + T i of the row, zeros past it).
template <int T, int CPT>
__device__ __forceinline__ float tree_sumsq(const float (&v)[CPT][16], float* s_part) {
  constexpr int L = kTreeLanes / T;  // tree lanes per thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int l = 0; l < L; ++l) {
    float acc = 0.0f;
#pragma unroll
    for (int i = l; i < CPT; i += L)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc = __fmaf_rn(v[i][j], v[i][j], acc);
#pragma unroll
    for (int o = 16; o; o >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, o));
    if (lane == 0) s_part[warp + (T / 32) * l] = acc;  // group of tree lanes 32 g .. 32 g + 31
  }
  __syncthreads();
  const float* p = s_part;
  return __fadd_rn(__fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3])),
                   __fadd_rn(__fadd_rn(p[4], p[5]), __fadd_rn(p[6], p[7])));
}

__device__ __forceinline__ float rms_factor(float ss, int K, float eps) {
  const float mean = __fdiv_rn(ss, static_cast<float>(K));
  return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(mean, eps)));
}

// Chunks of 16 bf16 factors (norm gains, gate rows), loaded ahead of their use.
template <int T, int CPT>
struct Factors {
  uint4 w[CPT][2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int chunks, bool wide) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = threadIdx.x + T * i;
      w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
      if (c < chunks) load_chunk(p + 16 * c, wide, w[i][0], w[i][1]);
    }
  }
};

// v[j] *= g[j].
__device__ __forceinline__ void mul_chunk(float* v, const uint4* w) {
  float g[16];
  unpack_bf16x8(w[0], g);
  unpack_bf16x8(w[1], g + 8);
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float2 r = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(g[j], g[j + 1]));
    v[j] = r.x;
    v[j + 1] = r.y;
  }
}

__device__ __forceinline__ void scale_chunk(float* v, float s) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float2 r = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(s, s));
    v[j] = r.x;
    v[j + 1] = r.y;
  }
}

// CTAs per SM that the register count is bounded for.  One chunk per thread:
// 48 registers and 1280 threads for bf16 outputs (4580 x 3584: 22.7 us; 24.2 at
// 60 registers), 64 and 1024 for FP8 ones, which spill at 48 (1024 x 3584: 10.6
// against 10.9 us).  Two chunks: 80 and 768 (4000 x 8192: 50 us, 62 unbounded).
// Four: 128 and 512 (1024 x 16384 bf16 34.7 us, 43.4 unbounded; 54 us with the
// eight chunks of the longest rows).  Eight: one CTA of 255.  All three residual
// forms of four and of eight chunks spill, 35 to 47 words a thread; 2000 x 12288
// to FP8 takes 56 us (3.1 TB/s), rotated 62.
constexpr int norm_min_ctas(int threads, int chunks, int out) {
  return chunks == 1 ? (out == 0 ? 1280 : 1024) / threads : chunks == 2 ? 768 / threads : chunks == 4 ? 2 : 1;
}

template <bool RESID, bool WHT, int OUT, int T, int CPT>
__global__ void __launch_bounds__(T, norm_min_ctas(T, CPT, OUT)) norm_rows_kernel(const NormArgs a) {
  __shared__ float s_part[2][kTreeLanes / 32];
  const int K = a.K, chunks = K >> 4;
  const int lane = threadIdx.x & 31;
  // the gate row loaded before the post norm's sum where its registers are
  // spare (1024 x 3584, FP8, a gate per row: 10.1 -> 9.6 us; 4580 rows bf16: 23.9 -> 25.0)
  constexpr bool kGateAhead = OUT == kOutFp8 && CPT == 1;
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    // plain loads of h and y: the outputs may overwrite them in place
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const __nv_bfloat16* h = a.h + row * K;
    uint4 hw[CPT][2];
    float v[CPT][16];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = threadIdx.x + T * i;
      hw[i][0] = hw[i][1] = zero;
      if (c < chunks) load_chunk(h + 16 * c, a.wide, hw[i][0], hw[i][1]);
    }
    if (RESID) {
      const __nv_bfloat16* y = a.y + row * K;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int c = threadIdx.x + T * i;
        uint4 y0 = zero, y1 = zero;
        if (c < chunks) load_chunk(y + 16 * c, a.wide, y0, y1);
        unpack_bf16x8(y0, v[i]);
        unpack_bf16x8(y1, v[i] + 8);
      }
      Factors<T, CPT> gate;
      if (kGateAhead && a.gate) gate.load(a.gate + (row / a.gate_rows) * K, chunks, a.wide);
      if (a.gamma_post) {
        Factors<T, CPT> g;
        g.load(a.gamma_post, chunks, a.wide);
        const float r = rms_factor(tree_sumsq<T, CPT>(v, s_part[0]), K, a.eps);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          scale_chunk(v[i], r);
          mul_chunk(v[i], g.w[i]);
        }
      }
      if (a.gate) {
        if (!kGateAhead) gate.load(a.gate + (row / a.gate_rows) * K, chunks, a.wide);
#pragma unroll
        for (int i = 0; i < CPT; ++i) mul_chunk(v[i], gate.w[i]);
      }
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int c = threadIdx.x + T * i;
        float hv[16];
        unpack_bf16x8(hw[i][0], hv);
        unpack_bf16x8(hw[i][1], hv + 8);
        // one at a time: a packed multiply and add would be joined to one rounding
#pragma unroll
        for (int j = 0; j < 16; ++j) v[i][j] = __fadd_rn(hv[j], __fmul_rn(v[i][j], a.alpha));
        if (c < chunks) store_chunk(a.h_out + row * K + 16 * c, a.wide, v[i]);
      }
      if (OUT == kOutBf16 && !a.x_out) {
        __syncthreads();  // the next row reuses s_part
        continue;
      }
    } else {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        unpack_bf16x8(hw[i][0], v[i]);
        unpack_bf16x8(hw[i][1], v[i] + 8);
      }
    }
    Factors<T, CPT> g;
    g.load(a.gamma_pre, chunks, a.wide);
    const float r = rms_factor(tree_sumsq<T, CPT>(v, s_part[1]), K, a.eps);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = threadIdx.x + T * i;
      scale_chunk(v[i], r);
      mul_chunk(v[i], g.w[i]);
      if (OUT == kOutBf16) {
        if (c < chunks) store_chunk(a.x_out + row * K + 16 * c, a.wide, v[i]);
      } else if ((c & ~31) < chunks) {  // warp-uniform
        if (WHT) wht64_lanes(v[i], lane);
        // a 1 x 128 block is on 8 adjacent lanes
        float m = fmaxf(absmax8(v[i]), absmax8(v[i] + 8));
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        const float s = row_global<1>(m);
        const Divisor dv = make_divisor(s);
        const uint2 lo = e4m3_codes8(v[i], dv), hi = e4m3_codes8(v[i] + 8, dv);
        if (c < chunks) {
          *reinterpret_cast<uint4*>(a.codes + row * K + 16 * c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
          if ((c & 7) == 0) a.scales[static_cast<int64_t>(c >> 3) * a.rows + row] = s;
        }
      }
    }
    __syncthreads();  // the next row reuses s_part
  }
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <bool RESID, bool WHT, int OUT, int T, int CPT>
cudaError_t launch_norm_shape(const NormArgs& a, cudaStream_t s) {
  // one row per CTA; very tall inputs loop (at most 64 CTAs per SM are launched)
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 64;
  const unsigned int grid = static_cast<unsigned int>(a.rows < cap ? a.rows : cap);
  return launch_pdl(norm_rows_kernel<RESID, WHT, OUT, T, CPT>, dim3(grid), dim3(T), 0, s, a);
}

template <bool RESID, bool WHT, int OUT>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  if (a.K <= 1024) return launch_norm_shape<RESID, WHT, OUT, 64, 1>(a, s);
  if (a.K <= 2048) return launch_norm_shape<RESID, WHT, OUT, 128, 1>(a, s);
  if (a.K <= 4096) return launch_norm_shape<RESID, WHT, OUT, 256, 1>(a, s);
  if (a.K <= 8192) return launch_norm_shape<RESID, WHT, OUT, 256, 2>(a, s);
  if (a.K <= 16384) return launch_norm_shape<RESID, WHT, OUT, 256, 4>(a, s);
  return launch_norm_shape<RESID, WHT, OUT, 256, 8>(a, s);
}

// Rotated 1 x 128 blocks of a call up to which they stay on 8 lanes per 64
// elements (more CTAs, shorter chains; spread / in threads, us, buffers larger
// than L2): 512 x 3584 (14336 blocks) 3.7 / 4.2, 1024 x 3584 (28672) 5.7 / 5.8,
// 8192 x 512 (32768) 6.1 / 6.0, 256 x 18944 (37888) 6.6 / 6.3, 1024 x 18944
// (151552) 21.7 / 14.7.
constexpr int64_t kFewBlocks = 30000;

// starve: boxes of half the rows, so that no tile ever has all its bytes and the
// wait for it runs out (the failure self test).
template <bool WEIGHT>
cudaError_t launch_rotated(const void* X, int64_t rows, int64_t K, uint8_t* codes, float* scales, bool starve,
                           cudaStream_t s) {
  CUtensorMap map, out_map;
  const uint64_t cols = static_cast<uint64_t>(K);
  if (!make_bf16_map(&map, X, cols, static_cast<uint64_t>(rows), starve ? 64 : 128) ||
      !make_map(&out_map, codes, cols, static_cast<uint64_t>(rows), cols, 128))
    return cudaErrorInvalidValue;
  RotArgs r;
  r.rows = rows;
  const int64_t k_blocks = (K + 127) / 128, tiles = (rows + 127) / 128 * k_blocks;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  r.k_blocks = static_cast<uint32_t>(k_blocks);
  r.tiles = static_cast<uint32_t>(tiles);
  r.scales = scales;
  r.budget = starve ? kStarvedBudgetCycles : kWaitBudgetCycles;
  const cudaError_t e = cudaFuncSetAttribute(quant_rotated_kernel<WEIGHT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kRotSmem);
  if (e != cudaSuccess) return e;
  const uint32_t ctas = 2 * static_cast<uint32_t>(device_sm_count());
  return launch_pdl(quant_rotated_kernel<WEIGHT>, dim3(r.tiles < ctas ? r.tiles : ctas), dim3(kRotThreads), kRotSmem, s,
                    map, out_map, r);
}

}  // namespace

cudaError_t launch_quant_act_fp8_block(const void* X, int64_t M, int64_t K, const void* gamma, float eps,
                                       uint32_t flags, uint8_t* codes, float* s_x, cudaStream_t s) {
  const bool wht = (flags & kFlagHadamard) != 0;
  if (flags & kFlagRmsNorm) {
    NormArgs a = {};
    a.h = static_cast<const __nv_bfloat16*>(X);
    a.gamma_pre = static_cast<const __nv_bfloat16*>(gamma);
    a.eps = eps;
    a.codes = codes;
    a.scales = s_x;
    a.rows = M;
    a.K = static_cast<int>(K);
    a.wide = aligned32(a.h) && aligned32(a.gamma_pre);
    return wht ? launch_norm<false, true, kOutFp8>(a, s) : launch_norm<false, false, kOutFp8>(a, s);
  }
  const int64_t blocks = (K + 127) / 128;
  if (wht && M * blocks > kFewBlocks) return launch_rotated<false>(X, M, K, codes, s_x, false, s);
  BlocksArgs a;
  a.X = static_cast<const __nv_bfloat16*>(X);
  a.rows = M;
  a.K = K;
  a.blocks = blocks;
  a.total = M * blocks;
  a.inv_blocks = blocks == 1 ? 0 : ~0ull / static_cast<unsigned long long>(blocks) + 1;
  a.codes = codes;
  a.scales = s_x;
  const int per_cta = wht ? kSpreadBlocks : kPlainBlocks;
  const int64_t grid = (a.total + per_cta - 1) / per_cta;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(wht ? quant_rotated_spread_kernel : quant_blocks_kernel, dim3(static_cast<unsigned int>(grid)),
                    dim3(kBlocksThreads), 0, s, a);
}

cudaError_t launch_quant_weight_fp8_block(const void* W, int64_t N, int64_t K, uint32_t flags, uint8_t* codes,
                                          float* s_w, cudaStream_t s) {
  if (flags & kFlagHadamard) return launch_rotated<true>(W, N, K, codes, s_w, false, s);
  const int64_t tiles = ((N + 127) / 128) * ((K + 127) / 128);
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(quant_weight_block_kernel, dim3(static_cast<unsigned int>(tiles)), dim3(kWeightThreads), 0, s,
                    static_cast<const __nv_bfloat16*>(W), N, K, codes, s_w);
}

cudaError_t launch_rotated_fp8_block(bool weight, bool starve, const void* X, int64_t rows, int64_t K, uint8_t* codes,
                                     float* scales, cudaStream_t s) {
  return weight ? launch_rotated<true>(X, rows, K, codes, scales, starve, s)
                : launch_rotated<false>(X, rows, K, codes, scales, starve, s);
}

cudaError_t block_quant_status_word(unsigned int** out) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(out), g_vlaq_block128_status);
}

cudaError_t launch_residual_norm(const ResidualNorm& r, cudaStream_t s) {
  NormArgs a = {};
  a.h = static_cast<const __nv_bfloat16*>(r.H);
  a.y = static_cast<const __nv_bfloat16*>(r.Y);
  a.gamma_post = static_cast<const __nv_bfloat16*>(r.gamma_post);
  a.gate = static_cast<const __nv_bfloat16*>(r.gate);
  a.gate_rows = r.gate_rows;
  a.alpha = r.alpha;
  a.gamma_pre = static_cast<const __nv_bfloat16*>(r.gamma_pre);
  a.eps = r.eps;
  a.h_out = static_cast<__nv_bfloat16*>(r.H_out);
  a.x_out = static_cast<__nv_bfloat16*>(r.X_out);
  a.codes = r.codes;
  a.scales = r.s_x;
  a.rows = r.M;
  a.K = static_cast<int>(r.K);
  a.wide = aligned32(a.h) && aligned32(a.y) && aligned32(a.gamma_post) && aligned32(a.gate) && aligned32(a.gamma_pre) &&
           aligned32(a.h_out) && aligned32(a.x_out);
  if (!r.codes) return launch_norm<true, false, kOutBf16>(a, s);
  return (r.flags & kFlagHadamard) ? launch_norm<true, true, kOutFp8>(a, s) : launch_norm<true, false, kOutFp8>(a, s);
}

}  // namespace vlaq
