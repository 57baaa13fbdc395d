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
// gemm_fp8_stream_kernel: the weights are the M = 128 operand, so that one
// weight scale belongs to the whole tile and block, and a tile of output
// channels is consecutive over the lanes when it is written; the tokens are N
// (16 to 128 at a time).  For few tokens the weights are the whole cost: the
// work (tiles x pairs of K blocks) is cut into one equal range for each SM
// whatever the tile count, so every SM streams the same number of weight bytes.
// A tile that several ranges share is summed by whichever of them arrives last,
// over the partial sums in the workspace in range order: the result does not
// depend on the schedule, and no second launch is needed.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/sga.h"
#include "sga_host.h"
#include "sga_internal.cuh"
#include "sga_ptx.cuh"

namespace sga {
namespace {

constexpr int kBlock = 128;  // K elements (bytes) and weight rows that share a scale

// ---------------------------------------------------------------- quantiser
constexpr int kQuantLanes = 16;  // threads per block of 128: 8 values (16 bytes) each

__device__ __forceinline__ uint32_t quantize4(uint32_t a, uint32_t b, float inv) {
  const float2 lo = make_float2(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv);
  const float2 hi = make_float2(__uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv);
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
         (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16);
}

// Half a warp per (token, block of 128 channels).  Bound by the 3 bytes per value it moves, and by the
// launch for the few tokens of a decode step.
__global__ void __launch_bounds__(256) quantize_fp8_kernel(const uint16_t* x, uint8_t* codes, float* scale, int cols,
                                                           int col_blocks, long long blocks) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int sub = threadIdx.x % kQuantLanes;
  const long long stride = static_cast<long long>(gridDim.x) * (256 / kQuantLanes);
  for (long long i = static_cast<long long>(blockIdx.x) * (256 / kQuantLanes) + threadIdx.x / kQuantLanes; i < blocks;
       i += stride) {
    const long long row = i / col_blocks;
    const int j = static_cast<int>(i - row * col_blocks);
    const int c = j * kBlock + 8 * sub;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < cols) v = __ldg(reinterpret_cast<const uint4*>(x + row * cols + c));  // cols is a multiple of 16
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    // the largest magnitude as bf16 bits, NaN (above 0x7F80) left out
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t lo = w[q] & 0x7FFFu, hi = (w[q] >> 16) & 0x7FFFu;
      if (lo <= 0x7F80u) top = max(top, lo);
      if (hi <= 0x7F80u) top = max(top, hi);
    }
#pragma unroll
    for (int o = kQuantLanes / 2; o > 0; o >>= 1)
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o, kQuantLanes));
    // top = 1.f * 2^(E - 127); 448 = 1.75 * 2^8
    int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
    e = top == 0 ? 0 : min(max(e, -126), 120);
    const uint2 o = make_uint2(quantize4(w[0], w[1], __uint_as_float(static_cast<uint32_t>(127 - e) << 23)),
                               quantize4(w[2], w[3], __uint_as_float(static_cast<uint32_t>(127 - e) << 23)));
    if (c < cols) *reinterpret_cast<uint2*>(codes + row * cols + c) = o;
    if (sub == 0) scale[i] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }
}

// ---------------------------------------------------------------- streaming product
constexpr int kTileM = 128;                     // weight rows per tile
constexpr int kWBytes = kTileM * kBlock;        // one K block of a weight tile: 16 KB
constexpr int kUnit = 2;                        // K blocks per ring stage
constexpr int kChunk = 16;                      // K blocks per scale slot
constexpr int kStreamThreads = 256;             // warps: TMA, MMA, 2 of scales, 4 of accumulation
constexpr int kAccBufs = 4;
constexpr int kMaxGrid = 148;                   // thread blocks (ranges); sizes the workspace
constexpr size_t kCounterOff = host::kStatusBytes;
constexpr size_t kPartOff = kCounterOff + 1024;
static_assert(kMaxGrid * 4 <= 1024, "counters");
static_assert(kPartOff + sizeof(float) * kMaxGrid * 2 * kTileM * 128 <= SGA_GEMM_FP8_WORKSPACE_BYTES, "workspace");

template <int NP>
struct StreamCfg {
  static constexpr int kXBytes = NP * kBlock;
  static constexpr int kStageBytes = kUnit * (kWBytes + kXBytes);
  static constexpr int kStages = NP <= 32 ? 5 : NP == 64 ? 4 : 3;
  static constexpr int kScaleBytes = 2 * kChunk * NP * 4;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 4 + 1;
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + kScaleBytes + kNumBars * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct StreamParams {
  int n, m, n_blocks, k_blocks, units;  // units: pairs of K blocks in a tile
  long long total;                      // units of all tiles
  const float* x_scale;
  const float* w_scale;
  float* out_f32;
  uint16_t* out_bf16;
  float* part;
  int* counters;
  int* status;
};

// One thread block's part of one tile: units [u0, u1) of `units`.
struct Segment {
  int mt, nb, u0, u1;
  long long tile;
};

__device__ __forceinline__ long long range_begin(const StreamParams& p, int c) { return p.total * c / gridDim.x; }

__device__ __forceinline__ Segment segment_at(const StreamParams& p, long long x, long long end) {
  Segment s;
  s.tile = x / p.units;
  s.u0 = static_cast<int>(x - s.tile * p.units);
  s.u1 = static_cast<int>(min(static_cast<long long>(p.units), s.u0 + (end - x)));
  s.nb = static_cast<int>(s.tile % p.n_blocks);
  s.mt = static_cast<int>(s.tile / p.n_blocks);
  return s;
}

template <int NP>
__global__ void __launch_bounds__(kStreamThreads, 1)
    gemm_fp8_stream_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                           StreamParams p) {
  using Cfg = StreamCfg<NP>;
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
  volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < kAccBufs; ++a) {
      mbar_init(accfull(a), 1);
      mbar_init(accempty(a), 4);  // one arrival per accumulating warp
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(sfull(a), 64);
      mbar_init(sempty(a), 4);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&wmap);
    prefetch_tmap(&xmap);
  }
  constexpr uint32_t kTmemCols = kAccBufs * NP;  // 64 .. 512
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();
  const long long begin = range_begin(p, blockIdx.x), end = range_begin(p, blockIdx.x + 1);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
      int st = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      for (long long x = begin; x < end && ok;) {
        const Segment sg = segment_at(p, x, end);
        for (int u = sg.u0; u < sg.u1; ++u) {
          if (!mbar_wait(empty(st), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const int nkb = min(kUnit, p.k_blocks - kUnit * u);
          mbar_arrive_expect_tx(full(st), nkb * (kWBytes + Cfg::kXBytes));
          const uint32_t dst = ring + st * Cfg::kStageBytes;
          for (int h = 0; h < nkb; ++h) {
            const int kb = kUnit * u + h;
            tma_load_2d(dst + h * kWBytes, &wmap, full(st), kb * kBlock, sg.mt * kTileM, pol_w);
            tma_load_2d(dst + kUnit * kWBytes + h * Cfg::kXBytes, &xmap, full(st), kb * kBlock, sg.nb * NP, pol_x);
          }
          ++issued;
          if (++st == Cfg::kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
        x += sg.u1 - sg.u0;
      }
      if (!ok) {
        record_status(p.status, kStatusTimeout);
        *abort_flag = 1;
        volatile int never = 0;
        for (long long i = (issued > Cfg::kStages ? issued - Cfg::kStages : 0); i < issued; ++i)
          mbar_wait(full(static_cast<int>(i % Cfg::kStages)), static_cast<uint32_t>((i / Cfg::kStages) & 1), &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kTileM, NP);
      int st = 0, buf = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (long long x = begin; x < end && ok;) {
        const Segment sg = segment_at(p, x, end);
        for (int u = sg.u0; u < sg.u1 && ok; ++u) {
          if (!mbar_wait(full(st), ph, abort_flag)) {
            ok = false;
            break;
          }
          const int nkb = min(kUnit, p.k_blocks - kUnit * u);
          const uint32_t a = ring + st * Cfg::kStageBytes;
          for (int h = 0; h < nkb; ++h) {
            if (!mbar_wait(accempty(buf), aph ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 K elements (bytes) per MMA
              mma_e4m3(tmem + buf * NP, sdesc_sw128(a + h * kWBytes + kk * 32, 16, 1024),
                       sdesc_sw128(a + kUnit * kWBytes + h * Cfg::kXBytes + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
            mma_commit(accfull(buf));
            if (++buf == kAccBufs) {
              buf = 0;
              aph ^= 1u;
            }
          }
          if (!ok) break;
          mma_commit(empty(st));
          if (++st == Cfg::kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
        x += sg.u1 - sg.u0;
      }
      if (!ok) {
        record_status(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      mma_commit(done_bar);
      volatile int never = 0;
      mbar_wait(done_bar, 0, &never);  // every MMA has finished before TMEM is freed
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ scales
    // Products x_scale * w_scale of up to 16 K blocks at a time, two slots.
    const int t = threadIdx.x - 64;
    int slot = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (long long x = begin; x < end && ok;) {
      const Segment sg = segment_at(p, x, end);
      const float* ws = p.w_scale + static_cast<size_t>(sg.mt) * p.k_blocks;
      for (int kb0 = kUnit * sg.u0; kb0 < kUnit * sg.u1; kb0 += kChunk) {
        if (!mbar_wait(sempty(slot), ph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        float* dst = scales + slot * kChunk * NP;
#pragma unroll 8
        for (int i = t; i < kChunk * NP; i += 64) {
          const int kbl = i % kChunk, tok = i / kChunk, kb = kb0 + kbl;
          const int token = sg.nb * NP + tok;
          float v = 0.f;
          if (kb < p.k_blocks && token < p.n)
            v = __ldg(p.x_scale + static_cast<size_t>(token) * p.k_blocks + kb) * __ldg(ws + kb);
          dst[kbl * NP + tok] = v;
        }
        mbar_arrive(sfull(slot));
        slot ^= 1;
        if (slot == 0) ph ^= 1u;
      }
      x += sg.u1 - sg.u0;
    }
    if (!ok) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------------ scaled accumulation
    // Warp w reads TMEM lane quarter w % 4: this thread's weight row is 32 (w % 4) + lane of the tile, its
    // accumulators are the NP tokens.
    const int quarter = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const int mrow = quarter * 32 + lane;
    int buf = 0, slot = 0;
    uint32_t aph = 0, sph = 0;
    bool ok = true;
    for (long long x = begin; x < end && ok;) {
      const Segment sg = segment_at(p, x, end);
      x += sg.u1 - sg.u0;
      float acc[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) acc[i] = 0.f;
      const int kb_end = min(kUnit * sg.u1, p.k_blocks);
      for (int kb0 = kUnit * sg.u0; kb0 < kb_end && ok; kb0 += kChunk) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(sfull(slot), sph, abort_flag));
        if (!ok) break;
        const float* sc = scales + slot * kChunk * NP;
        const int kb1 = min(kb0 + kChunk, kb_end);
        for (int kb = kb0; kb < kb1; ++kb, sc += NP) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(accfull(buf), aph, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint32_t src = tmem + lane_addr + buf * NP;
          constexpr int kCols = NP < 32 ? NP : 32;
#pragma unroll
          for (int c = 0; c < NP; c += kCols) {
            float v[kCols];
            if constexpr (kCols == 16) {
              tmem_ld16(src + c, v);
            } else {
              tmem_ld32(src + c, v);
            }
#pragma unroll
            for (int i = 0; i < kCols; i += 4) {
              const float4 s4 = *reinterpret_cast<const float4*>(sc + c + i);
              acc[c + i] = fmaf(v[i], s4.x, acc[c + i]);
              acc[c + i + 1] = fmaf(v[i + 1], s4.y, acc[c + i + 1]);
              acc[c + i + 2] = fmaf(v[i + 2], s4.z, acc[c + i + 2]);
              acc[c + i + 3] = fmaf(v[i + 3], s4.w, acc[c + i + 3]);
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
      ok = !named_barrier_or(1, 128, !ok);  // all four warps write, or none
      if (!ok) break;
      bool write = true;
      if (sg.u0 != 0 || sg.u1 != p.units) {
        // A shared tile: leave the partial sums, and let the last of the tile's ranges add them all in order.
        const long long t0 = sg.tile * p.units;
        const int c0 = static_cast<int>(((t0 + 1) * gridDim.x - 1) / p.total);            // range of its first unit
        const int c1 = static_cast<int>(((t0 + p.units) * gridDim.x - 1) / p.total);      // and of its last
        auto part_of = [&](int c) {
          const int second = range_begin(p, c) / p.units != sg.tile;  // a range's first tile, or its last
          return p.part + (static_cast<size_t>(2 * c + second) * NP) * kTileM + mrow;
        };
        float* mine = part_of(blockIdx.x);
#pragma unroll
        for (int i = 0; i < NP; ++i) mine[i * kTileM] = acc[i];
        __threadfence();
        named_barrier(1, 128);
        if (threadIdx.x == 128) {
          const int before = atomicAdd(p.counters + c0, 1);
          *last_flag = before == c1 - c0;
          if (before == c1 - c0) p.counters[c0] = 0;
          __threadfence();
        }
        named_barrier(1, 128);
        write = *last_flag != 0;
        if (write) {
#pragma unroll
          for (int i = 0; i < NP; ++i) acc[i] = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float* from = part_of(c);
#pragma unroll
            for (int i = 0; i < NP; ++i) acc[i] += __ldcg(from + i * kTileM);
          }
        }
        named_barrier(1, 128);  // last_flag read by all before the next tile writes it
      }
      const int row = sg.mt * kTileM + mrow;
      if (write && row < p.m) {
        const int tok0 = sg.nb * NP;
        const size_t at0 = static_cast<size_t>(tok0) * p.m + row;
        const int cols = min(NP, p.n - tok0);
        if (p.out_bf16) {
#pragma unroll
          for (int i = 0; i < NP; ++i)
            if (i < cols) p.out_bf16[at0 + static_cast<size_t>(i) * p.m] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i]));
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i)
            if (i < cols) p.out_f32[at0 + static_cast<size_t>(i) * p.m] = acc[i];
        }
      }
    }
    if (!ok) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int NP>
cudaError_t launch_stream(const GemmFp8Args& a, int num_sms, cudaStream_t s) {
  using Cfg = StreamCfg<NP>;
  StreamParams p;
  p.n = a.n;
  p.m = a.m;
  p.n_blocks = (a.n + NP - 1) / NP;
  p.k_blocks = (a.k + kBlock - 1) / kBlock;
  p.units = (p.k_blocks + kUnit - 1) / kUnit;
  p.total = static_cast<long long>((a.m + kTileM - 1) / kTileM) * p.n_blocks * p.units;
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.out_f32 = a.out_f32;
  p.out_bf16 = a.out_bf16;
  p.part = host::at<float>(a.ws, kPartOff);
  p.counters = host::at<int>(a.ws, kCounterOff);
  p.status = a.status;
  CUtensorMap wmap, xmap;
  cudaError_t e = make_tmap_2d(&wmap, true, a.w, a.k, a.m, a.k, kBlock, kTileM);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&xmap, true, a.x, a.k, a.n, a.k, kBlock, NP);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(gemm_fp8_stream_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(Cfg::kSmem));
  if (e != cudaSuccess) return e;
  const long long grid = std::min<long long>(std::min(num_sms, kMaxGrid), p.total);
  return host::launch_pdl(gemm_fp8_stream_kernel<NP>, dim3(static_cast<unsigned>(grid)), dim3(kStreamThreads),
                          Cfg::kSmem, s, wmap, xmap, p);
}

}  // namespace

cudaError_t launch_quantize_fp8(int rows, int cols, const uint16_t* x, uint8_t* codes, float* scale, cudaStream_t s) {
  const int col_blocks = (cols + kBlock - 1) / kBlock;
  const long long blocks = static_cast<long long>(rows) * col_blocks;
  const long long per = 256 / kQuantLanes;
  const long long grid = std::min<long long>((blocks + per - 1) / per, 148LL * 8);
  return host::launch_pdl(quantize_fp8_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, x, codes, scale,
                          cols, col_blocks, blocks);
}

cudaError_t launch_gemm_fp8(const GemmFp8Args& a, int num_sms, cudaStream_t s) {
  if (a.n <= 16) return launch_stream<16>(a, num_sms, s);
  if (a.n <= 32) return launch_stream<32>(a, num_sms, s);
  if (a.n <= 64) return launch_stream<64>(a, num_sms, s);
  return launch_stream<128>(a, num_sms, s);
}

}  // namespace sga

extern "C" {

sga_status_t sga_quantize_fp8(int32_t rows, int32_t cols, const sga_bf16_t* x, sga_fp8_e4m3_t* codes, float* scale,
                              sga_stream_t stream) {
  using sga::host::aligned;
  if (rows < 1 || cols < 16 || cols % 16 != 0) return SGA_ERR_INVALID_ARG;
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
  if (out_type != SGA_OUT_FP32 && out_type != SGA_OUT_BF16) return SGA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x_scale, 4) || !aligned(w, 16) || !aligned(w_scale, 4) ||
      !aligned(y, out_type == SGA_OUT_FP32 ? 4 : 2))
    return SGA_ERR_INVALID_ARG;
  if (!aligned(ws, sga::host::kWsAlign) || ws_bytes < SGA_GEMM_FP8_WORKSPACE_BYTES) return SGA_ERR_WORKSPACE;
  int sms = 0;
  const sga_status_t st = sga::host::device_info(&sms);
  if (st != SGA_OK) return st;
  sga::host::NvtxRange range("sga.gemm_fp8");
  sga::GemmFp8Args a{n, m, k, x, x_scale, w, w_scale, out_type == SGA_OUT_FP32 ? static_cast<float*>(y) : nullptr,
                     out_type == SGA_OUT_BF16 ? static_cast<uint16_t*>(y) : nullptr, ws, static_cast<int*>(ws)};
  return sga::host::from_cuda(sga::launch_gemm_fp8(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
