// Products with E4M3 operands that carry one fp32 scale for each block of 128
// (sga_gemm_fp8), and the quantiser that makes such activations
// (sga_quantize_fp8):
//
//   y[t][i] = sum_j xs[t][j] ws[i / 128][j] sum_{c in block j} x[t][c] w[i][c]
//
// The scales change with every block j of K, so a block's partial product (four
// tcgen05.mma kind::f8f6f4 of K = 32) lands in tensor memory of its own and is
// added to fp32 accumulators in registers with its scale, while the tensor core
// works on the next block.
//
// gemm_fp8_stream_kernel, few tokens or few tiles: the weights are the M = 128 operand, so that one weight scale belongs
// to the whole tile and block, and a thread's outputs are consecutive over the lanes; the tokens are N (16 to 128 at a
// time).  Bound by the weights' bytes, or where those are few by the latency of the chain (load, MMA, TMEM read, output).
// Where the tiles do not fill the SMs, K is split over a cluster whose thread blocks add up each other's partial sums
// through distributed shared memory, in a fixed order: the result does not depend on the schedule, and no second launch is
// needed.  (Sums in global memory by whichever block arrived last cost 4 to 6 us more.)  4 x 2304 x 7168 (n x m x k)
// 7.0 us, 2.4 TB/s; 32 x 20544 x 1536 8.6 us, 3.8 TB/s; 256 x 2304 x 7168 15.6 us.
//
// gemm_fp8_tile_kernel, many tokens: pairs of CTAs, 256 tokens x 256 channels a tile, the tokens as M.  Bound by the
// hand-over between the MMA (512 cycles a K block) and the scaled sums in registers (450 cycles) over two accumulators of
// 256 columns, and by power at large sizes: 4096 x 7168 x 8192 227 us on zeros, 264 on data, 1.8 PFLOP/s (the MMAs alone
// 147).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/sga.h"
#include "sga_host.h"
#include "sga_internal.cuh"
#include "sga_ptx.cuh"

namespace sga {
namespace {

constexpr int kBlock = 128;  // K elements (bytes) and weight rows that share a scale

// ---------------------------------------------------------------- pairs of scales past fp32's range
// Both kernels multiply a block's sum v by x_scale * w_scale.  Where that product is no normal fp32 number (it
// overflows, or loses bits as a subnormal or zero) v * x_scale * w_scale may still be one: v is zero or between 2^-18
// and 2^25 in magnitude (E4M3 products are multiples of 2^-18).  Such pairs are rare, and a branch in the accumulating
// loops costs 3% to 20% of the large products.  So the warps that fetch the scales only note that the thread block met
// one, and after its last tile it looks for the elements concerned and computes them once more, here.  An infinite
// product leaves an infinity or a NaN (also on v = 0).  A subnormal one is off by at most 2^-150, so its block by 2^-125:
// within fp32's rounding of any result from 2^-100 on.

// Zero, subnormal, infinite or NaN.
__device__ __forceinline__ bool not_normal(float s) {
  return (__float_as_uint(s) & 0x7FFFFFFFu) - 0x00800000u >= 0x7F000000u;
}

// The largest and the least magnitude but zero of the scales seen so far, as their bits (a NaN is the largest).
struct ScaleRange {
  uint32_t big = 0, small_1 = 0xFFFFFFFFu;  // the least, minus one: a zero is the largest there
  __device__ __forceinline__ void see(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
    big = max(big, b);
    small_1 = min(small_1, b - 1u);
  }
  // Whether one of them may have no normal product with w (those of zeros are zero, as they should be).
  __device__ __forceinline__ bool odd_with(float w) const {
    return w != 0.f && big != 0 &&
           (not_normal(__uint_as_float(big) * w) || not_normal(__uint_as_float(small_1 + 1u) * w));
  }
};

// The product as s * pre: pre is a power of two, v * pre is exact, and v * pre * s rounds once.
struct ScalePair {
  float s, pre;
};
__device__ __forceinline__ ScalePair scale_pair(float x, float w) {
  const float s = x * w;
  const float big = fmaxf(fabsf(x), fabsf(w)), small = fminf(fabsf(x), fabsf(w));
  // zeros and infinities are what they are; so is NaN (which fmaxf and fminf leave out)
  if (!not_normal(s) || isnan(s) || small == 0.f || isinf(big)) return {s, 1.f};
  if (fabsf(s) <= 1.f) return {copysignf(small * 0x1p100f * big, s), 0x1p-100f};
  // a rest of 2^128 and more times v is infinite for every v but zero, and so is FLT_MAX
  return {copysignf(fminf(big * 0x1p-100f * small, FLT_MAX), s), 0x1p100f};
}

__device__ __forceinline__ bool sure(float y) { return fabsf(y) >= 0x1p-100f && fabsf(y) <= FLT_MAX; }

__device__ __noinline__ bool any_odd_pair(const float* xs, const float* ws, int k_blocks) {
  bool odd = false;
#pragma unroll 1
  for (int kb = 0; kb < k_blocks; ++kb) odd |= scale_pair(xs[kb], ws[kb]).pre != 1.f;
  return odd;
}

// One output element, from its rows and their scales.
__device__ __noinline__ float scaled_dot(const uint8_t* x, const uint8_t* w, const float* xs, const float* ws, int k) {
  float acc = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < k; c0 += kBlock) {
    float v = 0.f;
#pragma unroll 1
    for (int c = c0; c < min(c0 + kBlock, k); c += 16) {  // k is a multiple of 16
      const uint4 a = *reinterpret_cast<const uint4*>(x + c), b = *reinterpret_cast<const uint4*>(w + c);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const auto pair = [&](const uint32_t (&q)[4]) {
          const auto two = static_cast<__nv_fp8x2_storage_t>(q[i >> 1] >> (16 * (i & 1)));
          return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
        };
        const float2 fa = pair(aw), fb = pair(bw);
        v = fmaf(fa.y, fb.y, fmaf(fa.x, fb.x, v));
      }
    }
    const ScalePair sp = scale_pair(xs[c0 / kBlock], ws[c0 / kBlock]);
    acc = fmaf(v * sp.pre, sp.s, acc);
  }
  return acc;
}

// ---------------------------------------------------------------- quantiser
constexpr int kQuantLanes = 16;  // threads per block of 128: 8 values (16 bytes) each

__device__ __forceinline__ uint32_t quantize4(uint32_t a, uint32_t b, float inv) {
  const float2 lo = make_float2(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv);
  const float2 hi = make_float2(__uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv);
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
         (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16);
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Half a warp per (token, block of 128 channels), kAhead blocks each: one where the launch counts, two where the
// bandwidth does (4096 x 8192: 18.6 us, 5.4 TB/s; one 19.9, four 21.5, and a grid of one wave that loops 21.5).
template <int kAhead>
__global__ void __launch_bounds__(256) quantize_fp8_kernel(const uint16_t* x, uint8_t* codes, float* scale, int cols,
                                                           int col_blocks, int blocks) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int sub = threadIdx.x % kQuantLanes;
  const int stride = gridDim.x * (256 / kQuantLanes);
  const bool whole = cols % kBlock == 0;  // then the blocks follow one another in memory
  const int i0 = blockIdx.x * (256 / kQuantLanes) + threadIdx.x / kQuantLanes;
  uint4 v[kAhead];
  size_t at[kAhead];
  bool in[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int i = i0 + u * stride;
    in[u] = i < blocks;
    v[u] = make_uint4(0, 0, 0, 0);
    if (whole) {
      at[u] = static_cast<size_t>(i) * kBlock + 8 * sub;
    } else {
      const int row = i / col_blocks, c = (i - row * col_blocks) * kBlock + 8 * sub;
      at[u] = static_cast<size_t>(row) * cols + c;
      in[u] &= c < cols;  // cols is a multiple of 16: a thread's eight values are in or out together
    }
    if (in[u]) v[u] = ld_stream16(x + at[u]);
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    // the largest magnitude as bf16 bits; where there is a NaN (above 0x7F80), again without it
    uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                            __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    top = max(top & 0xFFFFu, top >> 16);
    if (top > 0x7F80u) {
      top = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = w[q] & 0x7FFFu, hi = (w[q] >> 16) & 0x7FFFu;
        if (lo <= 0x7F80u) top = max(top, lo);
        if (hi <= 0x7F80u) top = max(top, hi);
      }
    }
#pragma unroll
    for (int o = kQuantLanes / 2; o > 0; o >>= 1)
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o, kQuantLanes));
    // top = 1.f * 2^(E - 127); 448 = 1.75 * 2^8
    int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
    e = top == 0 ? 0 : min(max(e, -126), 120);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    if (in[u]) *reinterpret_cast<uint2*>(codes + at[u]) = make_uint2(quantize4(w[0], w[1], inv), quantize4(w[2], w[3], inv));
    const int i = i0 + u * stride;
    if (sub == 0 && i < blocks) scale[i] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }
}

// ---------------------------------------------------------------- streaming product
constexpr int kTileM = 128;                     // weight rows per tile
constexpr int kWBytes = kTileM * kBlock;        // one K block of a weight tile: 16 KB
constexpr int kUnit = 2;                        // K blocks per ring stage
constexpr int kChunk = 16;                      // K blocks per scale slot
constexpr int kMaxSplits = 8;                   // thread blocks of a cluster

template <int NP>
struct StreamCfg {
  static constexpr int kXBytes = NP * kBlock;
  static constexpr int kStageBytes = kUnit * (kWBytes + kXBytes);
  static constexpr int kStages = NP <= 32 ? 5 : NP == 64 ? 4 : 3;
  static constexpr int kScaleBytes = 2 * kChunk * NP * 4;
  static constexpr int kAccBufs = NP <= 64 ? 4 : 2;  // accumulators of one unit: kUnit x NP columns
  // Warps: TMA, MMA, 2 of scales, then 4 or 8 of accumulation; of 8, four take each half of the tokens (an
  // accumulating warp's step is mostly the latency of its waits and loads, which the halves overlap).
  static constexpr int kGroups = NP >= 32 ? 2 : 1;
  static constexpr int kCols = NP / kGroups;
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 4 + 1;
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + kScaleBytes + kNumBars * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
  // the partial sums of a split tile, 128 rows x NP tokens, lie over the ring
  static_assert(kStages * kStageBytes >= 4 * kTileM * (NP + kMaxSplits), "receive buffer");
};

struct StreamParams {
  int n, m, k, n_blocks, tiles, k_blocks, units;  // tiles: 128 weight rows x NP tokens; units: pairs of K blocks in one
  int splits;                                     // thread blocks (a cluster) that share a tile's K
  const uint8_t* x;
  const uint8_t* w;
  const float* x_scale;
  const float* w_scale;
  float* out_f32;
  uint16_t* out_bf16;
  int* status;
  bool w_static;
};

// y[token0 + i * stride][row] = value(i) for i < count (at most kMost, unrolled).
template <int kMost, class Value>
__device__ __forceinline__ void store_y(const StreamParams& p, int row, int token0, int stride, int count,
                                        Value value) {
  const size_t at = static_cast<size_t>(token0) * p.m + row, step = static_cast<size_t>(stride) * p.m;
  if (p.out_bf16) {
    uint16_t* o = p.out_bf16 + at;
#pragma unroll
    for (int i = 0; i < kMost; ++i, o += step)
      if (i < count) *o = __bfloat16_as_ushort(__float2bfloat16_rn(value(i)));
  } else {
    float* o = p.out_f32 + at;
#pragma unroll
    for (int i = 0; i < kMost; ++i, o += step)
      if (i < count) *o = value(i);
  }
}

// y[token][row] as it was stored.
template <class Params>
__device__ __forceinline__ float load_y(const Params& p, int token, int row) {
  const size_t at = static_cast<size_t>(token) * p.m + row;
  return p.out_bf16 ? __uint_as_float(static_cast<uint32_t>(p.out_bf16[at]) << 16) : p.out_f32[at];
}

// Computes this thread's outputs of every tile of its thread block once more where a block's scales have no normal
// product.  (By itself, so that nothing of it is held in registers meanwhile.)
template <int NP>
__device__ __noinline__ void redo_stream_tiles(StreamParams p) {
  using Cfg = StreamCfg<NP>;
  const int warp = threadIdx.x >> 5, mrow = (warp & 3) * 32 + (threadIdx.x & 31), group = (warp - 4) >> 2;
  const int rank = blockIdx.x % p.splits;
  // the same thread wrote them
  const int c0 = p.splits == 1 ? group * Cfg::kCols : NP * rank / p.splits + group;
  const int c1 = p.splits == 1 ? c0 + Cfg::kCols : NP * (rank + 1) / p.splits;
  for (int t = blockIdx.x / p.splits; t < p.tiles; t += gridDim.x / p.splits) {
    const int row = t / p.n_blocks * kTileM + mrow, token0 = t % p.n_blocks * NP;
    if (row >= p.m) continue;
    const float* ws = p.w_scale + static_cast<size_t>(row / kBlock) * p.k_blocks;
    for (int i = token0 + c0; i < min(token0 + c1, p.n); i += p.splits == 1 ? 1 : Cfg::kGroups) {
      if (sure(load_y(p, i, row))) continue;
      const float* xs = p.x_scale + static_cast<size_t>(i) * p.k_blocks;
      if (!any_odd_pair(xs, ws, p.k_blocks)) continue;
      const float y = scaled_dot(p.x + static_cast<size_t>(i) * p.k, p.w + static_cast<size_t>(row) * p.k, xs, ws, p.k);
      store_y<1>(p, row, i, 0, 1, [&](int) { return y; });
    }
  }
}

template <int NP>
__global__ void __launch_bounds__(StreamCfg<NP>::kThreads, 1)
    gemm_fp8_stream_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                           StreamParams p) {
  using Cfg = StreamCfg<NP>;
  constexpr int kAccBufs = Cfg::kAccBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + Cfg::kStages * Cfg::kStageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kStages * Cfg::kStageBytes + Cfg::kScaleBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (Cfg::kStages + s); };
  auto accfull = [&](int a) { return bar0 + 8u * (2 * Cfg::kStages + a); };
  auto accempty = [&](int a) { return bar0 + 8u * (2 * Cfg::kStages + kAccBufs + a); };
  auto sfull = [&](int a) { return bar0 + 8u * (2 * Cfg::kStages + 2 * kAccBufs + a); };
  auto sempty = [&](int a) { return bar0 + 8u * (2 * Cfg::kStages + 2 * kAccBufs + 2 + a); };
  const uint32_t done_bar = bar0 + 8u * (2 * Cfg::kStages + 2 * kAccBufs + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* odd_scales = reinterpret_cast<volatile int*>(tmem_slot + 2);  // such a pair was met
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;
  // This thread block's tiles (token blocks fastest, so that neighbours share weights) and its part [u0, u1) of each
  // one's K.
  const int rank = blockIdx.x % p.splits;
  const int first = blockIdx.x / p.splits, step = gridDim.x / p.splits;
  const int u0 = p.units * rank / p.splits, u1 = p.units * (rank + 1) / p.splits;
  const int kb_end = min(kUnit * u1, p.k_blocks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < kAccBufs; ++a) {
      mbar_init(accfull(a), 1);
      mbar_init(accempty(a), 4 * Cfg::kGroups);  // one arrival per accumulating warp
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(sfull(a), 64);
      mbar_init(sempty(a), 4 * Cfg::kGroups);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    *odd_scales = 0;
    fence_barrier_init();
    prefetch_tmap(&wmap);
    prefetch_tmap(&xmap);
  }
  constexpr uint32_t kTmemCols = kAccBufs * kUnit * NP;  // 128 .. 512
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp != 0) {  // the producer waits in its own time
    grid_dependency_wait();
    grid_launch_dependents();
  }

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_w = p.n_blocks == 1 ? policy_evict_first() : policy_evict_last(), pol_x = policy_evict_last();
      const auto blocks_of = [&](int u) { return min(kUnit, p.k_blocks - kUnit * u); };
      auto load_w = [&](int st, int row0, int u) {
        const uint32_t dst = ring + st * Cfg::kStageBytes;
        for (int h = 0; h < blocks_of(u); ++h)
          tma_load_2d(dst + h * kWBytes, &wmap, full(st), (kUnit * u + h) * kBlock, row0, pol_w);
      };
      auto load_x = [&](int st, int token0, int u) {
        const uint32_t dst = ring + st * Cfg::kStageBytes + kUnit * kWBytes;
        for (int h = 0; h < blocks_of(u); ++h)
          tma_load_2d(dst + h * Cfg::kXBytes, &xmap, full(st), (kUnit * u + h) * kBlock, token0, pol_x);
      };
      // While the kernel before this one runs: weights that it cannot write are loaded into the first stages; others
      // are only brought into L2, which holds whatever it writes.
      int pre = 0;
      for (; pre < Cfg::kStages && u0 + pre < u1; ++pre) {
        if (p.w_static) {
          mbar_arrive_expect_tx(full(pre), blocks_of(u0 + pre) * (kWBytes + Cfg::kXBytes));
          load_w(pre, first / p.n_blocks * kTileM, u0 + pre);
        } else {
          for (int h = 0; h < blocks_of(u0 + pre); ++h)
            tma_prefetch_2d(&wmap, (kUnit * (u0 + pre) + h) * kBlock, first / p.n_blocks * kTileM);
        }
      }
      if (!p.w_static) pre = 0;
      grid_dependency_wait();
      grid_launch_dependents();
      int st = 0, n_done = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      for (int t = first; t < p.tiles && ok; t += step) {
        const int row0 = t / p.n_blocks * kTileM, token0 = t % p.n_blocks * NP;
        SGA_DCHECK(p.status, row0 < p.m && token0 < p.n && u0 < u1 && u1 <= p.units);
        for (int u = u0; u < u1; ++u, ++n_done) {
          if (n_done >= pre) {
            if (!mbar_wait(empty(st), ph ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(full(st), blocks_of(u) * (kWBytes + Cfg::kXBytes));
            load_w(st, row0, u);
          }
          load_x(st, token0, u);
          ++issued;
          if (++st == Cfg::kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        record_status(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // The copies in flight land before the ring is reused and the thread block exits, also when the MMA warp gave up.
      volatile int never = 0;
      for (long long i = (issued > Cfg::kStages ? issued - Cfg::kStages : 0); i < issued; ++i)
        mbar_wait(full(static_cast<int>(i % Cfg::kStages)), static_cast<uint32_t>((i / Cfg::kStages) & 1), &never);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    constexpr uint32_t idesc = idesc_e4m3_f32(kTileM, NP);
    const uint32_t acc = __shfl_sync(kAll, tmem, 0);
    int st = 0, buf = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true;
    for (int t = first; t < p.tiles && ok; t += step) {
      for (int u = u0; u < u1 && ok; ++u) {
        ok = mbar_wait_warp(full(st), ph, abort_flag) && mbar_wait_warp(accempty(buf), aph ^ 1u, abort_flag);
        if (!ok) break;
        const int nkb = min(kUnit, p.k_blocks - kUnit * u);
        const uint32_t a = ring + st * Cfg::kStageBytes;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < kUnit; ++h) {
            if (h < nkb) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 32 K elements (bytes) per MMA
                mma_e4m3(acc + (buf * kUnit + h) * NP, sdesc_sw128(a + h * kWBytes + kk * 32, 16, 1024),
                         sdesc_sw128(a + kUnit * kWBytes + h * Cfg::kXBytes + kk * 32, 16, 1024), idesc,
                         kk > 0 ? 1u : 0u);
            }
          }
          mma_commit(accfull(buf));
          mma_commit(empty(st));
        }
        __syncwarp();
        if (++buf == kAccBufs) {
          buf = 0;
          aph ^= 1u;
        }
        if (++st == Cfg::kStages) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
    if (elect_one()) mma_commit(done_bar);
    __syncwarp();
    volatile int never = 0;
    mbar_wait(done_bar, 0, &never);  // every MMA has finished before TMEM is freed and the ring reused
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ scales
    // Products x_scale * w_scale of up to 16 K blocks at a time, two slots.
    const int t64 = threadIdx.x - 64;
    int slot = 0;
    uint32_t ph = 0;
    bool ok = true, odd = false;
    for (int t = first; t < p.tiles && ok; t += step) {
      const float* ws = p.w_scale + static_cast<size_t>(t / p.n_blocks) * p.k_blocks;
      const int token0 = t % p.n_blocks * NP;
      for (int kb0 = kUnit * u0; kb0 < kb_end; kb0 += kChunk) {
        // this thread's K block and every fourth token, all loads before the first store (addresses past the end are
        // clamped: their products scale zeros or go unused)
        const int kbl = t64 % kChunk, tok0 = t64 / kChunk, kb = min(kb0 + kbl, p.k_blocks - 1);
        const float wv = __ldg(ws + kb);
        float v[NP / 4];
#pragma unroll
        for (int i = 0; i < NP / 4; ++i)
          v[i] = __ldg(p.x_scale + static_cast<size_t>(min(token0 + tok0 + 4 * i, p.n - 1)) * p.k_blocks + kb);
        if (!mbar_wait(sempty(slot), ph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        float* dst = scales + slot * kChunk * NP;
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) dst[kbl * NP + tok0 + 4 * i] = v[i] * wv;
        mbar_arrive(sfull(slot));
        ScaleRange range;
#pragma unroll
        for (int i = 0; i < NP / 4; ++i) range.see(v[i]);
        odd |= range.odd_with(wv);
        slot ^= 1;
        if (slot == 0) ph ^= 1u;
      }
    }
    if (!ok) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
    if (odd) *odd_scales = 1;
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scaled accumulation
    // Warp w reads TMEM lane quarter w % 4: this thread's weight row is 32 (w % 4) + lane of the tile, its
    // accumulators are the tokens col0 .. col0 + kCols - 1.
    constexpr int kCols = Cfg::kCols;
    const int quarter = warp & 3, col0 = ((warp - 4) >> 2) * kCols;
    const uint32_t src0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
    const int mrow = quarter * 32 + lane;
    int buf = 0, slot = 0;
    uint32_t aph = 0, sph = 0;
    bool ok = true;
    float acc[kCols];
    const auto add = [&](const float* v, const float* sc) {
#pragma unroll
      for (int i = 0; i < kCols; i += 4) {
        const float4 s4 = *reinterpret_cast<const float4*>(sc + i);
        acc[i] = fmaf(v[i], s4.x, acc[i]);
        acc[i + 1] = fmaf(v[i + 1], s4.y, acc[i + 1]);
        acc[i + 2] = fmaf(v[i + 2], s4.z, acc[i + 2]);
        acc[i + 3] = fmaf(v[i + 3], s4.w, acc[i + 3]);
      }
    };
    for (int t = first; t < p.tiles && ok; t += step) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
      for (int kb0 = kUnit * u0; kb0 < kb_end && ok; kb0 += kChunk) {
        ok = mbar_wait_warp(sfull(slot), sph, abort_flag);
        if (!ok) break;
        const float* sc = scales + slot * kChunk * NP + col0;
        const int kb1 = min(kb0 + kChunk, kb_end);
        for (int kb = kb0; kb < kb1; kb += kUnit, sc += kUnit * NP) {
          ok = mbar_wait_warp(accfull(buf), aph, abort_flag);
          if (!ok) break;
          tc_fence_after();
          // both K blocks of the unit (the second one's columns go unused past the last K block)
          const uint32_t src = src0 + buf * kUnit * NP;
          const bool two = kb + 1 < kb1;
          if constexpr (kCols <= 32) {
            float v[2 * kCols];
            if constexpr (kCols == 16) {
              tmem_ld16x2(src, src + NP, v);
            } else {
              tmem_ld32x2(src, src + NP, v);
            }
            add(v, sc);
            if (two) add(v + kCols, sc + NP);
          } else {
            float v[kCols];
            tmem_ld64(src, v);
            add(v, sc);
            if (two) {
              tmem_ld64(src + NP, v);
              add(v, sc + NP);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(accempty(buf));
          if (++buf == kAccBufs) {
            buf = 0;
            aph ^= 1u;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty(slot));
        slot ^= 1;
        if (slot == 0) sph ^= 1u;
      }
      const int row = t / p.n_blocks * kTileM + mrow, token0 = t % p.n_blocks * NP + col0;
      if (ok && p.splits == 1 && row < p.m)
        store_y<kCols>(p, row, token0, 1, p.n - token0, [&](int i) { return acc[i]; });
    }
    if (!ok && lane == 0) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
    __syncwarp();
    if (p.splits > 1) {
      // A tile shared by the cluster (its only one): thread block r sums tokens c0(r) .. c0(r + 1) - 1, c0(r) = NP r / S,
      // over the ranks in order.  Each sends its partial sums of those tokens to r, into the idle ring, as
      // [source][token][128 rows].
      const int S = p.splits, width = (NP + S - 1) / S;
      const uint32_t inv = 65536u / S + 1;  // x / S = x * inv >> 16 for x <= 8 NP
      const auto c0_of = [&](int r) { return static_cast<int>((static_cast<uint32_t>(NP * r) * inv) >> 16); };
      cluster_barrier();  // every MMA of the cluster has finished
      const uint32_t mine = ring + 4u * (rank * width * kTileM + mrow);
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = col0 + i, r = ((c + 1) * S - 1) / NP;  // the r with c0(r) <= c < c0(r + 1)
        SGA_DCHECK(p.status, r < S && c0_of(r) <= c && c < c0_of(r + 1) && c - c0_of(r) < width);
        st_cluster(map_to_rank(mine + 4u * (c - c0_of(r)) * kTileM, r), acc[i]);
      }
      cluster_barrier();
      const int c0 = c0_of(rank), c1 = c0_of(rank + 1);
      const int row = first / p.n_blocks * kTileM + mrow, token0 = first % p.n_blocks * NP;
      const float* part = reinterpret_cast<const float*>(smem) + mrow;
      if (ok && row < p.m) {
        // this warp's half of the tokens, eight at a time: their partial sums loaded together
        const int last = min(c1, p.n - token0);
        for (int i0 = c0 + (warp - 4) / 4; i0 < last; i0 += 8 * Cfg::kGroups) {
          float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int r = 0; r < S; ++r) {
#pragma unroll
            for (int q = 0; q < 8; ++q)  // past the last token: any of the buffer's values
              sum[q] += part[(r * width + min(i0 + q * Cfg::kGroups, last - 1) - c0) * kTileM];
          }
          store_y<8>(p, row, token0 + i0, Cfg::kGroups, (last - i0 + Cfg::kGroups - 1) / Cfg::kGroups,
                     [&](int q) { return sum[q]; });
        }
      }
    }
  }
  if (warp < 4 && p.splits > 1) {
    cluster_barrier();
    // the thread blocks that write the tile's output have to know
    if ((warp == 2 || warp == 3) && lane < p.splits && *odd_scales)
      st_cluster(map_to_rank(smem_u32(tmem_slot + 2), lane), __uint_as_float(1u));
    cluster_barrier();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (*odd_scales && !*abort_flag && warp >= 4) redo_stream_tiles<NP>(p);
}

// What the kernel takes for `tiles` tiles of NP tokens, in microseconds, and the split of K it takes it with.  Fitted to
// runs of 1 to 8 splits at 300 x 2048, 300 x 8192 and 1900 x 4096 weights with 8, 32, 64 and 96 tokens: a unit 0.43 (16
// tokens) to 0.85 us (128 tokens), an exchange 1 to 3 us and 0.3 us for each thread block that joins it, another
// tile's output 2 us.  300 x 2048, 8
// tokens: 5.6 us unsplit, 4.4 in four, 4.4 in eight; 300 x 8192: 15.8, 6.9, 5.5.  Only splits whose clusters all run at
// once are considered.
struct StreamPlan {
  int splits;
  float us;
};
StreamPlan stream_plan(int np, long long tiles, int units) {
  const float unit = 0.42f + 0.000026f * np * np;
  const float base = 2.3f + 0.004f * np;
  const float waves = static_cast<float>((tiles + 147) / 148);
  StreamPlan best = {1, base + unit * static_cast<float>(units) * waves + 2.f * (waves - 1.f)};
  for (int splits = 2; splits <= kMaxSplits && splits <= units; ++splits) {
    if (tiles > host::kClusters[splits - 1]) break;
    const float us = base + unit * static_cast<float>((units + splits - 1) / splits) + 0.1f + 0.0185f * np +
                     0.3f * static_cast<float>(splits);
    if (us < best.us) best = {splits, us};
  }
  return best;
}

template <int NP>
cudaError_t launch_stream(const GemmFp8Args& a, int num_sms, cudaStream_t s) {
  using Cfg = StreamCfg<NP>;
  StreamParams p;
  p.n = a.n;
  p.m = a.m;
  p.k = a.k;
  p.x = a.x;
  p.w = a.w;
  p.n_blocks = (a.n + NP - 1) / NP;
  const long long tiles = static_cast<long long>((a.m + kTileM - 1) / kTileM) * p.n_blocks;
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  p.k_blocks = (a.k + kBlock - 1) / kBlock;
  p.units = (p.k_blocks + kUnit - 1) / kUnit;
  p.splits = stream_plan(NP, tiles, p.units).splits;
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.out_f32 = a.out_f32;
  p.out_bf16 = a.out_bf16;
  p.status = a.status;
  p.w_static = a.w_static;
  CUtensorMap wmap, xmap;
  cudaError_t e = make_tmap_2d(&wmap, true, a.w, a.k, a.m, a.k, kBlock, kTileM);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&xmap, true, a.x, a.k, a.n, a.k, kBlock, NP);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_fp8_stream_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(Cfg::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.splits > 1 ? p.tiles * p.splits : std::min(num_sms, p.tiles)));
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_fp8_stream_kernel<NP>, wmap, xmap, p);
}

// ---------------------------------------------------------------- tiled product (many tokens)
constexpr int kTM = 128;                       // tokens per CTA: half of MMA M, one token per TMEM lane
constexpr int kTN = 256;                       // output channels per tile: MMA N, two weight scale blocks
constexpr int kTStages = 4;                    // even: the two MMA warps take every other stage
constexpr int kTXBytes = kTM * kBlock;         // one K block of this CTA's tokens: 16 KB
constexpr int kTWBytes = kTN / 2 * kBlock;     // one K block of this CTA's half of the weights: 16 KB
constexpr int kTStageBytes = kTXBytes + kTWBytes;
constexpr int kTChunk = 8;                     // K blocks per scale slot
constexpr int kTScaleLd = kTM + 1;             // odd: the transposing stores of the scales hit distinct banks
constexpr int kTScaleFloats = kTChunk * kTScaleLd + 2 * kTChunk;
constexpr int kTThreads = 384;                 // warps: TMA, MMA (even K blocks, odd ones), scales, 8 of accumulation
constexpr int kTNumBars = 2 * kTStages + 4 + 4 + 2;
constexpr int kTOutFloats = 32 * 33;           // one accumulating warp's 32 x 32 transpose for the output
constexpr size_t kTSmem =
    1024 + kTStages * kTStageBytes + (2 * kTScaleFloats + 8 * kTOutFloats) * 4 + kTNumBars * 8 + 16;
static_assert(kTSmem <= 232448, "shared memory budget");
// Registers at launch: 384 threads x 168 = 64,512, shared out as 128 x 64 + 256 x 216.  (With 56 and 224 the compiler
// spills 100 bytes where the scales' range is kept, and a large product takes 8% longer.)
constexpr int kTRegsSmall = 64, kTRegsLarge = 216;
static_assert(128 * kTRegsSmall + 256 * kTRegsLarge <= 384 * 168, "register split");

struct TileParams {
  int n, m, k, n_tiles, m_tiles, k_blocks, tiles;
  const uint8_t* x;
  const uint8_t* w;
  const float* x_scale;
  const float* w_scale;
  float* out_f32;
  uint16_t* out_bf16;
  int* status;
  bool pair_stores;  // every even channel of out_bf16 lies on a 4-byte boundary
};

// (a, b) += (x, y) * s, two lanes an instruction.
__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float s) {
  asm("{\n\t.reg .b64 c, v, t;\n\t"
      "mov.b64 c, {%0, %1};\n\t"
      "mov.b64 v, {%2, %3};\n\t"
      "mov.b64 t, {%4, %4};\n\t"
      "fma.rn.f32x2 c, v, t, c;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y), "f"(s));
}

// As redo_stream_tiles: a warp takes its 32 tokens one by one, a lane every 32nd of its 128 channels.
__device__ __noinline__ void redo_tiles(TileParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3, half = (warp - 4) >> 2;
  for (int t = blockIdx.x >> 1; t < p.tiles; t += gridDim.x >> 1) {
    const int token0 = (2 * (t % p.n_tiles) + (blockIdx.x & 1)) * kTM + quarter * 32;
    const int ch0 = t / p.n_tiles * kTN + half * kBlock;
    const float* ws = p.w_scale + static_cast<size_t>(ch0 / kBlock) * p.k_blocks;
    for (int token = token0; token < min(token0 + 32, p.n); ++token) {
      const float* xs = p.x_scale + static_cast<size_t>(token) * p.k_blocks;
      for (int ch = ch0 + lane; ch < min(ch0 + kBlock, p.m); ch += 32) {
        if (sure(load_y(p, token, ch)) || !any_odd_pair(xs, ws, p.k_blocks)) continue;
        const float y = scaled_dot(p.x + static_cast<size_t>(token) * p.k, p.w + static_cast<size_t>(ch) * p.k, xs, ws, p.k);
        const size_t at = static_cast<size_t>(token) * p.m + ch;
        if (p.out_bf16) {
          p.out_bf16[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        } else {
          p.out_f32[at] = y;
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kTThreads, 1)
    gemm_fp8_tile_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                         TileParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + kTStages * kTStageBytes);
  float* out_stage = scales + 2 * kTScaleFloats;
  uint64_t* bars = reinterpret_cast<uint64_t*>(out_stage + 8 * kTOutFloats);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kTStages + s); };
  auto accfull = [&](int a) { return bar0 + 8u * (2 * kTStages + a); };
  auto accempty = [&](int a) { return bar0 + 8u * (2 * kTStages + 2 + a); };
  auto sfull = [&](int a) { return bar0 + 8u * (2 * kTStages + 4 + a); };
  auto sempty = [&](int a) { return bar0 + 8u * (2 * kTStages + 6 + a); };
  auto done = [&](int a) { return bar0 + 8u * (2 * kTStages + 8 + a); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kTNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* odd_scales = reinterpret_cast<volatile int*>(tmem_slot + 2);  // such a pair was met
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kTStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accfull(a), 1);
      mbar_init(accempty(a), 16);  // one arrival per accumulating warp of both CTAs (the leader's is used)
      mbar_init(sfull(a), 32);
      mbar_init(sempty(a), 8);
      mbar_init(done(a), 1);
    }
    *abort_flag = 0;
    *odd_scales = 0;
    fence_barrier_init();
    prefetch_tmap(&wmap);
    prefetch_tmap(&xmap);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // both CTAs' barriers are initialised before either signals the other
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  // Tiles go over the pairs with the tokens fastest: the pairs at work share few weight tiles and re-read the
  // tokens, which the L2 holds.
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTRegsSmall));
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      if (lane == 0) {
        const uint64_t pol = policy_evict_last();
        int st = 0;
        uint32_t ph = 0;
        long long issued = 0;
        bool ok = true;
        for (int t = pair; t < p.tiles && ok; t += pairs) {
          const int tn = t % p.n_tiles, tm = t / p.n_tiles;
          SGA_DCHECK(p.status, 2 * tn * kTM < p.n && tm * kTN < p.m);
          for (int kb = 0; kb < p.k_blocks; ++kb) {
            if (!mbar_wait_idle(empty(st), ph ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            // both CTAs' loads complete on the leader's barrier
            if (rank == 0) mbar_arrive_expect_tx(full(st), 2 * kTStageBytes);
            const uint32_t dst = ring + st * kTStageBytes;
            tma_load_2d_pair(dst, &xmap, full(st) & kPairLeaderMask, kb * kBlock, (2 * tn + rank) * kTM, pol);
            tma_load_2d_pair(dst + kTXBytes, &wmap, full(st) & kPairLeaderMask, kb * kBlock,
                             tm * kTN + rank * (kTN / 2), pol);
            ++issued;
            if (++st == kTStages) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        // The leader's last arrivals on this CTA's `empty` barriers have landed before the CTA may exit.
        for (int i = 0; i < kTStages && ok; ++i) {
          ok = mbar_wait_idle(empty(st), ph ^ 1u, abort_flag);
          if (++st == kTStages) {
            st = 0;
            ph ^= 1u;
          }
        }
        if (!ok) {
          record_status(p.status, kStatusTimeout);
          *abort_flag = 1;
        }
        // The copies in flight land before the pair exits, also when an MMA warp gave up (the peer waits for the leader
        // at the cluster barrier below).
        volatile int never = 0;
        if (rank == 0)
          for (long long i = (issued > kTStages ? issued - kTStages : 0); i < issued; ++i)
            mbar_wait_idle(full(static_cast<int>(i % kTStages)), static_cast<uint32_t>((i / kTStages) & 1), &never);
      }
    } else if (warp < 3) {
      // ---------------------------------------------------------- MMA issuers (of the leader, for both CTAs)
      // Two warps take every other K block of the pair's sequence and one accumulator each: a warp's waits for its
      // next block run while the other's block is in the tensor core (issuing a block takes nearly as long as
      // computing it, and the waits ~300 cycles more).
      if (rank == 0) {
        constexpr uint32_t kAll = 0xFFFFFFFFu;
        constexpr uint32_t idesc = idesc_e4m3_f32(2 * kTM, kTN);
        const int buf = warp - 1;
        const uint32_t acc = __shfl_sync(kAll, tmem, 0) + buf * kTN;
        const int my_tiles = (p.tiles - pair + pairs - 1) / pairs;
        const long long blocks = static_cast<long long>(my_tiles) * p.k_blocks;
        int st = buf;
        uint32_t ph = 0, aph = 0;
        bool ok = true;
        for (long long i = buf; i < blocks; i += 2) {
          ok = mbar_wait_idle_warp(full(st), ph, abort_flag) && mbar_wait_idle_warp(accempty(buf), aph ^ 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t a = ring + st * kTStageBytes;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 K elements (bytes) per MMA
              mma_e4m3_pair(acc, sdesc_sw128(a + kk * 32, 16, 1024), sdesc_sw128(a + kTXBytes + kk * 32, 16, 1024),
                            idesc, kk > 0 ? 1u : 0u);
            mma_commit_pair(accfull(buf));
            mma_commit_pair(empty(st));
          }
          __syncwarp();
          st += 2;  // the ring has an even number of stages
          if (st >= kTStages) {
            st -= kTStages;
            ph ^= 1u;
          }
          aph ^= 1u;
        }
        if (!ok && lane == 0) {
          record_status(p.status, kStatusTimeout);
          *abort_flag = 1;
        }
        if (elect_one()) mma_commit_pair_here(done(buf));
        __syncwarp();
        volatile int never = 0;
        mbar_wait_idle(done(buf), 0, &never);  // every MMA has finished before TMEM is freed
      }
    } else {
      // ---------------------------------------------------------- scales
      // Token scales of up to 8 K blocks at a time, transposed to [K block][token], and the two weight scales.
      const int m_blocks = (p.m + kBlock - 1) / kBlock;
      int slot = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = pair; t < p.tiles && ok; t += pairs) {
        const int tn = t % p.n_tiles, tm = t / p.n_tiles;
        for (int kb0 = 0; kb0 < p.k_blocks; kb0 += kTChunk) {
          if (!mbar_wait_idle(sempty(slot), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          float* dst = scales + slot * kTScaleFloats;
          // 16 loads before their stores (addresses past the end are clamped, their values dropped)
          const int kbl = lane % kTChunk, tok0 = lane / kTChunk, kb = kb0 + kbl;
          const float* col = p.x_scale + min(kb, p.k_blocks - 1);
          // the lane's K block of the channel blocks 2 tm and 2 tm + 1
          const float* wrow = p.w_scale + static_cast<size_t>(2 * tm) * p.k_blocks + min(kb, p.k_blocks - 1);
          const float w0 = __ldg(wrow), w1 = 2 * tm + 1 < m_blocks ? __ldg(wrow + p.k_blocks) : 0.f;
          ScaleRange range;
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            const int tok1 = tok0 + part * (kTM / 2);
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[i] = __ldg(col + static_cast<size_t>(min((2 * tn + rank) * kTM + tok1 + 4 * i, p.n - 1)) * p.k_blocks);
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[kbl * kTScaleLd + tok1 + 4 * i] = v[i];
#pragma unroll
            for (int i = 0; i < 16; ++i) range.see(v[i]);
          }
          if (lane < kTChunk) {
            dst[kTChunk * kTScaleLd + lane] = w0;
            dst[kTChunk * kTScaleLd + kTChunk + lane] = w1;
          }
          if (range.odd_with(w0) || range.odd_with(w1)) *odd_scales = 1;
          mbar_arrive(sfull(slot));
          slot ^= 1;
          if (slot == 0) ph ^= 1u;
        }
      }
      if (!ok) {
        record_status(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTRegsLarge));
    // ------------------------------------------------------------ scaled accumulation
    // Warp w: lane quarter w % 4 (token 32 (w % 4) + lane), the 128 channels of scale block `half`.
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t src0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kBlock;
    const int tok = quarter * 32 + lane;
    int buf = 0, slot = 0;
    uint32_t aph = 0, sph = 0;
    bool ok = true;
    for (int t = pair; t < p.tiles && ok; t += pairs) {
      const int tn = t % p.n_tiles, tm = t / p.n_tiles;
      float acc[kBlock];
#pragma unroll
      for (int i = 0; i < kBlock; ++i) acc[i] = 0.f;
      for (int kb0 = 0; kb0 < p.k_blocks && ok; kb0 += kTChunk) {
        ok = mbar_wait_idle_warp(sfull(slot), sph, abort_flag);
        if (!ok) break;
        const float* sc = scales + slot * kTScaleFloats;
        const int kbs = min(kTChunk, p.k_blocks - kb0);
        float s_next = sc[tok] * sc[kTChunk * kTScaleLd + half * kTChunk];
        for (int kbl = 0; kbl < kbs; ++kbl) {
          const float s = s_next;
          if (kbl + 1 < kbs) s_next = sc[(kbl + 1) * kTScaleLd + tok] * sc[kTChunk * kTScaleLd + half * kTChunk + kbl + 1];
          ok = mbar_wait_idle_warp(accfull(buf), aph, abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kBlock; c += 32) {
            float v[32];
            tmem_ld32(src0 + buf * kTN + c, v);
            if (c + 32 == kBlock) {  // all of this warp's columns are in registers
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(accempty(buf) & kPairLeaderMask);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) fma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], s);
          }
          buf ^= 1;
          if (buf == 0) aph ^= 1u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty(slot));
        slot ^= 1;
        if (slot == 0) sph ^= 1u;
      }
      // Output: 32 x 32 pieces turned over in shared memory, so that a store covers 32 consecutive channels of a token
      // whatever the alignment of its row.
      const int token0 = (2 * tn + rank) * kTM + quarter * 32, ch0 = tm * kTN + half * kBlock;
      const int rows = min(32, p.n - token0);
      if (!ok || rows <= 0) continue;
      float* stage = out_stage + (warp - 4) * kTOutFloats;
#pragma unroll
      for (int c = 0; c < kBlock; c += 32) {
        if (ch0 + c >= p.m) break;
#pragma unroll
        for (int i = 0; i < 32; ++i) stage[lane * 33 + i] = acc[c + i];
        __syncwarp();
        const int ch = ch0 + c + lane;
        if (p.pair_stores) {  // two tokens a store, two channels a lane
          const int pair_ch = ch0 + c + 2 * (lane & 15);
          uint16_t* o = p.out_bf16 + static_cast<size_t>(token0 + (lane >> 4)) * p.m + pair_ch;
#pragma unroll 8
          for (int r = 0; r < 32; r += 2, o += 2 * static_cast<size_t>(p.m)) {
            const float* v = stage + (r + (lane >> 4)) * 33 + 2 * (lane & 15);
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[0], v[1]);
            if (r + (lane >> 4) < rows && pair_ch < p.m) *reinterpret_cast<__nv_bfloat162*>(o) = b;
          }
        } else if (ch < p.m) {
          const size_t at0 = static_cast<size_t>(token0) * p.m + ch;
#pragma unroll 8
          for (int r = 0; r < rows; ++r) {
            const float v = stage[r * 33 + lane];
            if (p.out_bf16) {
              p.out_bf16[at0 + static_cast<size_t>(r) * p.m] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            } else {
              p.out_f32[at0 + static_cast<size_t>(r) * p.m] = v;
            }
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
    if (ok && *odd_scales) redo_tiles(p);
  }

  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // the pair's MMAs, copies and arrivals are done in both CTAs
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

cudaError_t launch_tile(const GemmFp8Args& a, int num_sms, cudaStream_t s) {
  TileParams p;
  p.n = a.n;
  p.m = a.m;
  p.k = a.k;
  p.x = a.x;
  p.w = a.w;
  p.n_tiles = (a.n + 2 * kTM - 1) / (2 * kTM);
  p.m_tiles = (a.m + kTN - 1) / kTN;
  p.k_blocks = (a.k + kBlock - 1) / kBlock;
  const long long tiles = static_cast<long long>(p.n_tiles) * p.m_tiles;
  if (tiles > INT32_MAX - num_sms) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.out_f32 = a.out_f32;
  p.out_bf16 = a.out_bf16;
  p.status = a.status;
  p.pair_stores = host::aligned(a.out_bf16, 4) && a.m % 2 == 0;
  CUtensorMap wmap, xmap;
  cudaError_t e = make_tmap_2d(&wmap, true, a.w, a.k, a.m, a.k, kBlock, kTN / 2);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&xmap, true, a.x, a.k, a.n, a.k, kBlock, kTM);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_fp8_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kTSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(num_sms / 2, p.tiles)));
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = kTSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_fp8_tile_kernel, wmap, xmap, p);
}

}  // namespace

cudaError_t launch_quantize_fp8(int rows, int cols, const uint16_t* x, uint8_t* codes, float* scale, cudaStream_t s) {
  const int col_blocks = (cols + kBlock - 1) / kBlock;
  const long long blocks = static_cast<long long>(rows) * col_blocks;
  if (blocks > kMaxExtent) return cudaErrorInvalidValue;
  constexpr int per = 256 / kQuantLanes;
  const int n = static_cast<int>(blocks);
  if (n <= 148 * 8 * per)  // one wave
    return host::launch_pdl(quantize_fp8_kernel<1>, dim3((n + per - 1) / per), dim3(256), 0, s, x, codes, scale, cols,
                            col_blocks, n);
  return host::launch_pdl(quantize_fp8_kernel<2>, dim3((n + 2 * per - 1) / (2 * per)), dim3(256), 0, s, x, codes, scale,
                          cols, col_blocks, n);
}

cudaError_t launch_gemm_fp8(const GemmFp8Args& a, int num_sms, cudaStream_t s) {
  if (a.n <= 16) return launch_stream<16>(a, num_sms, s);
  if (a.n <= 32) return launch_stream<32>(a, num_sms, s);
  if (a.n <= 64) return launch_stream<64>(a, num_sms, s);
  // More tokens: blocks of 128 through the streaming kernel, whose split K or smaller tiles fill the SMs where there are
  // few, or tiles of 256 x 256, which read the operands less often (a K block 0.45 us, another tile's output 5 us).
  // n x m x k, streaming against tiles: 256 x 2304 x 7168 15.6 us against 33, 512 x 4096 x 4096 17.7 against 21.5;
  // 700 x 4096 x 4096 31.9 against 21.5, 400 x 7168 x 8192 58.6 against 37.
  const long long k_blocks = (a.k + kBlock - 1) / kBlock;
  const long long m128 = (a.m + kTileM - 1) / kTileM, n128 = (a.n + 127) / 128;
  const long long waves = (((a.m + kTN - 1) / kTN) * static_cast<long long>((a.n + 2 * kTM - 1) / (2 * kTM)) + 73) / 74;
  const float tile_us = 7.f + 0.45f * static_cast<float>(k_blocks * waves) + 5.f * static_cast<float>(waves - 1);
  if (stream_plan(128, m128 * n128, static_cast<int>((k_blocks + kUnit - 1) / kUnit)).us < tile_us)
    return launch_stream<128>(a, num_sms, s);
  return launch_tile(a, num_sms, s);
}

}  // namespace sga

extern "C" {

sga_status_t sga_quantize_fp8(int32_t rows, int32_t cols, const sga_bf16_t* x, sga_fp8_e4m3_t* codes, float* scale,
                              sga_stream_t stream) {
  using sga::host::aligned;
  if (rows < 1 || cols < 16 || cols % 16 != 0 || cols > sga::kMaxExtent) return SGA_ERR_INVALID_ARG;
  if (static_cast<long long>(rows) * ((cols + sga::kBlock - 1) / sga::kBlock) > sga::kMaxExtent) return SGA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return SGA_ERR_INVALID_ARG;
  int sms = 0;
  const sga_status_t st = sga::host::device_info(&sms);
  if (st != SGA_OK) return st;
  sga::host::NvtxRange range("sga.quantize_fp8");
  return sga::host::from_cuda(
      sga::launch_quantize_fp8(rows, cols, x, codes, scale, static_cast<cudaStream_t>(stream)));
}

sga_status_t sga_gemm_fp8(int32_t n, int32_t m, int32_t k, const sga_fp8_e4m3_t* x, const float* x_scale,
                          const sga_fp8_e4m3_t* w, const float* w_scale, void* y, sga_out_type_t out_type, void* ws,
                          size_t ws_bytes, sga_stream_t stream) {
  using sga::host::aligned;
  if (n < 1 || m < 1 || k < 16 || k % 16 != 0) return SGA_ERR_INVALID_ARG;
  if (n > sga::kMaxExtent || m > sga::kMaxExtent || k > sga::kMaxExtent) return SGA_ERR_INVALID_ARG;
  if (out_type != SGA_OUT_FP32 && out_type != SGA_OUT_BF16) return SGA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x_scale, 4) || !aligned(w, 16) || !aligned(w_scale, 4) ||
      !aligned(y, out_type == SGA_OUT_FP32 ? 4 : 2))
    return SGA_ERR_INVALID_ARG;
  if (!aligned(ws, sga::host::kWsAlign) || ws_bytes < sga::host::kStatusBytes) return SGA_ERR_WORKSPACE;
  int sms = 0;
  const sga_status_t st = sga::host::device_info(&sms);
  if (st != SGA_OK) return st;
  sga::host::NvtxRange range("sga.gemm_fp8");
  sga::GemmFp8Args a{n, m, k, x, x_scale, w, w_scale, out_type == SGA_OUT_FP32 ? static_cast<float*>(y) : nullptr,
                     out_type == SGA_OUT_BF16 ? static_cast<uint16_t*>(y) : nullptr, static_cast<int*>(ws)};
  return sga::host::from_cuda(sga::launch_gemm_fp8(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
