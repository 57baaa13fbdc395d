// Sparse MLA attention over a latent cache held in 4 bits, then the head-specific
// sigmoid gate: the formulas of sga_attend.cu on rows of 416 bytes (512 E2M1
// codes, an E4M3 scale for each 16 of them, 64 bf16 rope values; see
// sga_sparse_mla_attend_kv4 in sga.h).
//
//   S = Q C^T * 192^-0.5,  P = softmax_s(S),  out = (P C[:, 0:512]) * sigmoid(g)
//
// What differs from the bf16 kernel follows from the row being 2.8 times smaller:
//   * A chunk's 64 rows are 26 KB, so they are gathered into registers: eight
//     producer warps hold the next two chunks' codes while they expand and store
//     the current one, and the whole value ring in shared memory is left to expanded tiles.
//   * A code times its scale has at most 6 significant bits between 2^-10 and
//     2,688, so it is exact in fp16 (and in bf16).  The tiles hold fp16: two
//     codes expand with one conversion and one multiplication, and P can be one
//     fp16 operand (half a step is 2^-11, an eighth of the rounding of the bf16
//     result) where the bf16 kernel needs two bf16 parts: half the PV
//     instructions.
//   * Q must then be fp16 for the latent dims.  Each head is scaled by the power
//     of two that takes its largest value into [2^14, 2^15): a bf16 value keeps
//     its 8 bits exactly down to 2^-31 of the head's largest, and the factor
//     is taken out again in the softmax scale.  (The scaled scores stay finite
//     for cache rope values up to 2^106: 64 products below 2^15 * 2^106.)  The rope dims stay bf16 on both
//     sides (kind::f16 takes either type, one per instruction).
// Otherwise as there: one CTA per (query, split), the splits of a query a cluster;
// QK^T with M = 64 heads, N = 64 rows; PV transposed, O^T [512 x 64] in tensor
// memory; a lazy running maximum in the log2 domain; the splits merged through
// distributed shared memory.
//
// Bound by the shared memory's 128 bytes a cycle: a chunk's products read 240 KB of
// operands (1,900 cycles), its tiles and P are 72 KB of stores, and a chunk takes
// 2,600 cycles.  512 queries of 2,048 slots: 198 us (146 GFLOP, 0.74 PFLOP/s).  Few queries
// are bound by the chain of one chunk after another and by the merge (128 KB per CTA
// over the distributed shared memory, 19 bytes a cycle): 4 queries 15.9 us, 32 queries
// over 32,768 positions 26.2 us.  Measured and left out: eight softmax warps (a
// wave of 148 queries 78 us against 52), two groups of them by turns (a fifth slower),
// waits by one lane of a warp (84 us), loads predicated and not branched around (56 us).
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include "sga_host.h"
#include "sga_internal.cuh"
#include "sga_ptx.cuh"

namespace cg = cooperative_groups;

namespace sga {
namespace {

constexpr int kHeads = 64;
constexpr int kDq = 576;
constexpr int kDv = 512;
constexpr int kChunk = 64;                   // selected rows per chunk
constexpr int kBoxBytes = kChunk * 128;      // 64 rows x 64 dims of 16 bits
constexpr int kPairBytes = 2 * kBoxBytes;    // 64 rows x 128 dims: A of one PV product
constexpr int kHalfBytes = 2 * kPairBytes;   // 64 rows x 256 dims, filled and released together
constexpr int kHalves = 2;                   // value dims 0..511
constexpr int kRing = 2 * kHalves;           // two chunks of value tiles
constexpr int kRopeRing = 2;
constexpr int kQBox = kHeads * 128;          // 64 heads x 64 dims
constexpr int kQBytes = 9 * kQBox;
constexpr int kPBytes = kHeads * kChunk * 2;  // 64 heads x 64 rows fp16
constexpr int kMaskRing = 4;
constexpr int kProducerWarps = 8;            // warps 0-7: four threads per chunk row
constexpr int kQkWarp = 8;                   // warps 8 and 9 issue QK^T of every other chunk
constexpr int kPvWarp = 10;                  // issues PV
constexpr int kSoftmaxWarp = 11;             // warps 11-14
constexpr int kSoftmaxThreads = 128;
constexpr int kThreads = 32 * kSoftmaxWarp + kSoftmaxThreads;
constexpr int kTmemCols = 512;
constexpr int kSCol = 256;
// barriers: full[4] empty[4] rope_full[2] rope_empty[2] q_full s_full[2] s_free[2]
//           p_full p_free o_full qk_done
constexpr int kNumBars = 2 * kRing + 2 * kRopeRing + 1 + 2 + 2 + 4;
constexpr int kMaxSplits = 8;                // splits of a query = CTAs of its cluster
constexpr size_t kSmemBytes = 1024 + kRing * kHalfBytes + kRopeRing * kBoxBytes + kQBytes + kPBytes +
                              kNumBars * 8 + kMaskRing * 8 + 2 * kHeads * 4 + kHeads * 8 + 16;
constexpr float kRescaleThreshold = 8.0f;    // log2 units
// P = 2^(x - max + 7): with a maximum that lags by at most 8 it stays within 2^15 and inside fp16, and fp16's
// smallest step is 2^-31 of the largest weight (the factor 2^7 is in O and in l alike and cancels).
constexpr float kPShift = 7.0f;
constexpr int kRowBytes = SGA_KV4_ROW_BYTES;
constexpr int kScaleOff = kDv / 2;           // byte offset of a row's scales
constexpr int kRopeOff = kScaleOff + kDv / 16;

static_assert(kRowBytes == kRopeOff + 2 * (kDq - kDv), "cache row layout");
static_assert(kSmemBytes <= 232448, "shared memory budget");
// the split merge's receive buffer lies over the value ring, the rope slots and the Q buffer (see sga_attend.cu)
static_assert(kRing * kHalfBytes + kRopeRing * kBoxBytes + kQBytes >= 7 * kHeads * 76 * 4,
              "split merge receive buffer");

struct Attend4Params {
  const uint16_t* q;
  const uint8_t* kv4;
  const int32_t* idx;
  const uint16_t* gate;
  uint16_t* out;
  int* status;
  int row0, n_q, kv_stride, top_k, splits, chunks;  // row0: the first query (of batch x n_q) of this launch
  float scale_log2;
};

__device__ __forceinline__ float sigmoidf_(float g) { return 1.0f / (1.0f + expf(-g)); }

// 2^x with the hardware approximation (relative error ~2^-22; results below
// 2^-126 flush to zero, which only drops weights far below the fp32 sum).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (a, b) = (a, b) * s + c, and (a, b) += (x, y): two lanes an instruction.
__device__ __forceinline__ void fma2(float& a, float& b, float s, float c) {
  asm("{\n\t.reg .b64 v, t, u;\n\t"
      "mov.b64 v, {%0, %1};\n\t"
      "mov.b64 t, {%2, %2};\n\t"
      "mov.b64 u, {%3, %3};\n\t"
      "fma.rn.f32x2 v, v, t, u;\n\t"
      "mov.b64 {%0, %1}, v;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(s), "f"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 v, t;\n\t"
      "mov.b64 v, {%0, %1};\n\t"
      "mov.b64 t, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, t;\n\t"
      "mov.b64 {%0, %1}, v;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32, 16 or 8 bytes, read once per query: volatile keeps the load where it is issued, ahead of its use.
__device__ __forceinline__ void ld_row32(const uint8_t* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ uint4 ld_row16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_row8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Four 8 x 8 blocks of 16-bit values in the fragment layout, to the rows whose addresses lanes 0-31 give.
__device__ __forceinline__ void stmatrix_x4(uint32_t row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two E4M3 scales (the low 16 bits) -> each of them in both halves of an fp16 pair.
__device__ __forceinline__ void expand_scales(uint32_t two, uint32_t& s0, uint32_t& s1) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
  s0 = __byte_perm(h, h, 0x1010);
  s1 = __byte_perm(h, h, 0x3232);
}

// Eight E2M1 codes (code 2j in the low half of byte j) times one scale -> eight fp16 values (exact).
__device__ __forceinline__ uint4 expand_codes(uint32_t codes, uint32_t scale) {
  uint4 v;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "r"(codes));
  v.x = hmul2(v.x, scale);
  v.y = hmul2(v.y, scale);
  v.z = hmul2(v.z, scale);
  v.w = hmul2(v.w, scale);
  return v;
}

// The part of one cache row that one of its four producer threads (part = 0..3) expands: 64 codes of each half (the
// half's box `part`), eight scales (exchanged among the four threads) and 16 rope values.
struct RowPart {
  uint4 codes[kHalves][2];
  uint2 scales;
  uint4 rope[2];
};

__device__ __forceinline__ void load_row(RowPart& d, const uint8_t* row, int part, bool valid) {
  if (valid) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) ld_row32(row + 128 * h + 32 * part, d.codes[h][0], d.codes[h][1]);
    d.scales = ld_row8(row + kScaleOff + 8 * part);
    ld_row32(row + kRopeOff + 32 * part, d.rope[0], d.rope[1]);
  } else {  // an empty slot: zeros (masked out of the softmax)
#pragma unroll
    for (int h = 0; h < kHalves; ++h) d.codes[h][0] = d.codes[h][1] = make_uint4(0, 0, 0, 0);
    d.scales = make_uint2(0, 0);
    d.rope[0] = d.rope[1] = make_uint4(0, 0, 0, 0);
  }
}

// The part of a query head that one of eight threads converts: column `part` of the head's row in the nine boxes.
struct QPart {
  uint4 v[9];
};

__device__ __forceinline__ void load_q(QPart& d, const uint16_t* q, int row, int head, int part) {
  const uint8_t* src = reinterpret_cast<const uint8_t*>(q) + (static_cast<size_t>(row) * kHeads + head) * kDq * 2 + 16 * part;
#pragma unroll
  for (int i = 0; i < 9; ++i) d.v[i] = ld_row16(src + 128 * i);
}

__device__ __forceinline__ void store_q(const QPart& d, uint32_t q_s, float* q_scale, int head, int part, float scale_log2) {
  uint32_t top = 0;  // largest magnitude as bf16 bits
#pragma unroll
  for (int i = 0; i < 9; ++i) {
    const uint32_t w[4] = {d.v[i].x, d.v[i].y, d.v[i].z, d.v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
  }
  top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  // 2^e takes a largest value of exponent x to exponent 14; heads smaller than 2^-86 have logits of zero anyway
  int e = 14 + 127 - static_cast<int>(top >> 7);
  e = top == 0 ? 0 : min(max(e, -113), 100);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
  for (int i = 0; i < 9; ++i) {
    const uint32_t w[4] = {d.v[i].x, d.v[i].y, d.v[i].z, d.v[i].w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = __uint_as_float(w[k] << 16) * up, hi = __uint_as_float(w[k] & 0xFFFF0000u) * up;
      o[k] = i < kDv / 64 ? pack_f16(lo, hi) : pack_bf16(lo, hi);  // the last box holds the rope dims
    }
    st_shared16(q_s + i * kQBox + head * 128 + ((part ^ (head & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
  }
  if (part == 0) q_scale[head] = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

__global__ void __launch_bounds__(kThreads, 1) sga_attend4_kernel(Attend4Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t pairs = smem_u32(smem);
  const uint32_t rope = pairs + kRing * kHalfBytes;
  const uint32_t q_s = rope + kRopeRing * kBoxBytes;
  const uint32_t p_s = q_s + kQBytes;
  uint8_t* p_ptr = smem + kRing * kHalfBytes + kRopeRing * kBoxBytes + kQBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(p_ptr + kPBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kRing + s); };
  auto rope_full = [&](int s) { return bar0 + 8u * (2 * kRing + s); };
  auto rope_empty = [&](int s) { return bar0 + 8u * (2 * kRing + kRopeRing + s); };
  const uint32_t q_full = bar0 + 8u * (2 * kRing + 2 * kRopeRing);
  auto s_full = [&](int b) { return q_full + 8u * (1 + b); };
  auto s_free = [&](int b) { return q_full + 8u * (3 + b); };
  const uint32_t p_full = q_full + 8u * 5;
  const uint32_t p_free = q_full + 8u * 6;
  const uint32_t o_full = q_full + 8u * 7;   // every PV MMA has finished
  const uint32_t qk_done = q_full + 8u * 8;  // every QK^T MMA has finished
  uint64_t* masks = bars + kNumBars;
  float* head_f = reinterpret_cast<float*>(masks + kMaskRing);  // [64] per-head factors
  float* q_scale = head_f + kHeads;                              // [64] softmax scale (log2) of the scaled heads
  float2* own_ml = reinterpret_cast<float2*>(q_scale + kHeads);  // [64] (m, l) of this split, read by the cluster
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(own_ml + kHeads);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int row = p.row0 + blockIdx.x / p.splits;
  const int split = static_cast<int>(cluster.block_rank());  // the cluster is the query's p.splits CTAs
  const int chunk0 = p.chunks * split / p.splits;            // at most 32 chunks, at least one per split
  const int nchunks = p.chunks * (split + 1) / p.splits - chunk0;
  const int slot_base = chunk0 * kChunk;                     // first selected slot of this split

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(full(s), kProducerWarps);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < kRopeRing; ++s) {
      mbar_init(rope_full(s), kProducerWarps);
      mbar_init(rope_empty(s), 1);
    }
    mbar_init(q_full, kProducerWarps + kSoftmaxThreads / 32);
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(s_free(b), kSoftmaxThreads / 32);
    }
    mbar_init(p_full, kSoftmaxThreads / 32);
    mbar_init(p_free, 1);
    mbar_init(o_full, 1);
    mbar_init(qk_done, 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Set-up above overlaps the previous kernel on the stream; every input is read below.
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp < kProducerWarps) {
    // ------------------------------------------------------------ gather and expansion
    const int b = row / p.n_q;
    const int32_t* idx_row = p.idx + static_cast<size_t>(row) * p.top_k;
    const uint8_t* kv_b = p.kv4 + static_cast<size_t>(b) * p.kv_stride * kRowBytes;
    const int ptid = threadIdx.x;
    const int r = ptid >> 2;    // this thread's row of the chunk
    const int part = ptid & 3;  // and its quarter of that row
    bool ok = true;
    // Rows are loaded two chunks ahead, at the end of an iteration, so that they have a whole one to arrive; their
    // indices are fetched one iteration before that.
    auto load_idx = [&](int j) {
      // K is a multiple of 64: a chunk has no tail
      SGA_DCHECK(p.status, j >= nchunks || (slot_base >= 0 && slot_base + j * kChunk + r < p.top_k));
      return j < nchunks ? __ldg(idx_row + slot_base + j * kChunk + r) : -1;
    };
    auto load = [&](RowPart& d, int v) {
      const bool valid = v >= 0 && v < p.kv_stride;
      if (!valid && v != -1) record_status(p.status, kStatusDeviceArg);
      load_row(d, kv_b + static_cast<size_t>(valid ? v : 0) * kRowBytes, part, valid);
      return valid;
    };
    const int first_idx = load_idx(0), second_idx = load_idx(1);
    int ahead_idx = load_idx(2);
    RowPart cur, next;
    bool cur_valid, next_valid = false;
    {
      // Q: this warp's four of the heads 0-31 (the softmax warps take the others)
      QPart v;
      load_q(v, p.q, row, 4 * warp + (lane >> 3), lane & 7);
      cur_valid = load(cur, first_idx);
      store_q(v, q_s, q_scale, 4 * warp + (lane >> 3), lane & 7, p.scale_log2);
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    if (nchunks > 1) next_valid = load(next, second_idx);
    // This thread's 64 dims of a half are the eight 16-byte columns of a row of box `part`, stored in the order
    // i ^ 2 part, so that the eight threads of a store phase (two rows) reach eight different columns.
    const uint32_t dst0 = pairs + part * kBoxBytes + r * 128 + (((2 * part) ^ (r & 7)) << 4);
    const uint32_t scale_order = 0x3210u ^ (0x1111u * part);
    for (int j = 0; j < nchunks; ++j) {
      const uint32_t seen = __ballot_sync(0xFFFFFFFFu, cur_valid);
      const int rs = j % kRopeRing;
      ok = mbar_wait_warp(rope_empty(rs), static_cast<uint32_t>((j / kRopeRing) & 1) ^ 1u, abort_flag);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        st_shared16(rope + rs * kBoxBytes + r * 128 + (((2 * part + i) ^ (r & 7)) << 4), cur.rope[i]);
      __syncwarp();
      if (lane == 0) {
        // Validity of the warp's eight rows (every fourth ballot bit) -> bits 8 warp .. of the chunk's mask, which
        // the softmax reads after S, so after this arrival.  Slot j % 4 is free: this warp has filled the pairs
        // of chunk j - 1, which PV(j - 3) had to release.
        uint32_t m = seen & 0x11111111u;
        m = (m | (m >> 3)) & 0x03030303u;
        m = (m | (m >> 6)) & 0x000F000Fu;
        m = (m | (m >> 12)) & 0xFFu;
        reinterpret_cast<uint8_t*>(masks + j % kMaskRing)[warp] = static_cast<uint8_t>(m);
        mbar_arrive(rope_full(rs));
      }
      // Value dims 256 half .. 256 half + 255 -> slot (2 j + half) mod 4: the first half is expanded in registers before its
      // slot is free, the other while QK^T reads the first.
#pragma unroll
      for (int half = 0; half < kHalves; ++half) {
        // the scales of box `part` are word 4 half + part of the row's eight: with thread (4 half + part) / 2
        const int from = (lane & ~3) + 2 * half + (part >> 1);
        const uint32_t w0 = __shfl_sync(0xFFFFFFFFu, cur.scales.x, from);
        const uint32_t w1 = __shfl_sync(0xFFFFFFFFu, cur.scales.y, from);
        const uint32_t four = __byte_perm((part & 1) ? w1 : w0, 0, scale_order);  // in the order of the columns
        uint32_t s[4];
        expand_scales(four & 0xFFFFu, s[0], s[1]);
        expand_scales(four >> 16, s[2], s[3]);
        const uint4 a = cur.codes[half][0], b = cur.codes[half][1];
        const bool f2 = part & 1, f4 = part & 2;
        const uint32_t t[8] = {f2 ? a.z : a.x, f2 ? a.w : a.y, f2 ? a.x : a.z, f2 ? a.y : a.w,
                               f2 ? b.z : b.x, f2 ? b.w : b.y, f2 ? b.x : b.z, f2 ? b.y : b.w};
        uint4 tile[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) tile[i] = expand_codes(f4 ? t[i ^ 4] : t[i], s[i >> 1]);
        const int n = j * kHalves + half;
        const int slot = n % kRing;
        ok = ok && mbar_wait_warp(empty(slot), static_cast<uint32_t>((n / kRing) & 1) ^ 1u, abort_flag);
        if (ok) {
          const uint32_t dst = dst0 + slot * kHalfBytes;
#pragma unroll
          for (int i = 0; i < 8; ++i) st_shared16(dst ^ (i << 4), tile[i]);
          __syncwarp();
          if (lane == 0) mbar_arrive(full(slot));
        }
      }
      if (!ok) break;
      cur = next;
      cur_valid = next_valid;
      if (j + 2 < nchunks) {
        next_valid = load(next, ahead_idx);
        ahead_idx = load_idx(j + 3);
      }
    }
    if (!ok) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
  } else if (warp < kSoftmaxWarp) {
    // ------------------------------------------------------------ MMA issuers
    // Two warps issue QK^T, every other chunk each, and one PV, each waiting on its own operands only: an issue lasts as
    // long as the products, and the waits of the next chunk run meanwhile.  The tiles, Q and P come from ordinary
    // stores: they are made visible to the tensor core here, between the wait for them and the MMA (the same fence in
    // the storing warps would also wait for the rows they have in flight).  Shared-memory descriptors differ in
    // their low words only, by the address over 16 (see sdesc_sw128).
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    const uint32_t acc = __shfl_sync(kAll, tmem, 0);
    const auto desc_lo = [](uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); };
    const auto desc = [](uint32_t lo) { return (sdesc_sw128(0, 0, 1024) & 0xFFFFFFFF00000000ull) | lo; };
    bool ok = true;
    if (warp < kPvWarp) {
      constexpr uint32_t idesc_lat = idesc_f16_f32(kHeads, kChunk, false, false);
      constexpr uint32_t idesc_rope = idesc_bf16_f32(kHeads, kChunk, false, false);
      const uint32_t q_lo = desc_lo(q_s, 16), pair_lo = desc_lo(pairs, 16), rope_lo = desc_lo(rope, 16);
      ok = mbar_wait_warp(q_full, 0, abort_flag);
      for (int j = warp - kQkWarp; j < nchunks && ok; j += 2) {
        const int sb = j & 1, rs = j % kRopeRing;
        const uint32_t d = acc + kSCol + sb * kChunk;
        ok = mbar_wait_warp(s_free(sb), static_cast<uint32_t>((j >> 1) & 1) ^ 1u, abort_flag) &&
             mbar_wait_warp(rope_full(rs), static_cast<uint32_t>((j / kRopeRing) & 1), abort_flag);
        // the rope box and the first half, then the second one, whose stores overlap the first one's products
        for (int half = 0; half < kHalves && ok; ++half) {
          const int n = j * kHalves + half;
          const int slot = n % kRing;
          ok = mbar_wait_warp(full(slot), static_cast<uint32_t>((n / kRing) & 1), abort_flag);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          if (elect_one()) {
            if (half == 0) {
              const uint32_t src = rope_lo + rs * (kBoxBytes >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16(d, desc(q_lo + 8 * (kQBox >> 4) + kk * 2), desc(src + kk * 2), idesc_rope, kk > 0 ? 1u : 0u);
              mma_commit(rope_empty(rs));  // rope dims are not needed for P V
            }
            const uint32_t src = pair_lo + slot * (kHalfBytes >> 4);
            const uint32_t qa = q_lo + 4 * half * (kQBox >> 4);
#pragma unroll
            for (int kk = 0; kk < 16; ++kk)  // four steps in each of the half's boxes
              mma_bf16(d, desc(qa + (kk >> 2) * (kQBox >> 4) + (kk & 3) * 2),
                       desc(src + (kk >> 2) * (kBoxBytes >> 4) + (kk & 3) * 2), idesc_lat, 1u);
            if (half == 1) mma_commit(s_full(sb));
          }
          __syncwarp();
        }
        ok = __all_sync(kAll, ok);
      }
    } else {
      constexpr uint32_t idesc_pv = idesc_f16_f32(128, kHeads, true, false);
      const uint32_t p_lo = desc_lo(p_s, 16), v_lo = desc_lo(pairs, kBoxBytes);
      for (int j = 0; j < nchunks; ++j) {
        ok = mbar_wait_warp(p_full, static_cast<uint32_t>(j & 1), abort_flag);
        if (!ok) break;
        fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          // O^T[dims 128 q ..][heads] += V^T P^T, one accumulator block per value pair
#pragma unroll
          for (int q = 0; q < 2 * kHalves; ++q) {
            const int slot = (j * kHalves + (q >> 1)) % kRing;
            const uint32_t v = v_lo + slot * (kHalfBytes >> 4) + (q & 1) * (kPairBytes >> 4);
            const uint32_t d = acc + q * kHeads;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // A = V^T: M = 128 dims over the pair's two boxes, K = rows 16 kk ..
              mma_bf16(d, desc(v + kk * (2048 >> 4)), desc(p_lo + kk * 2), idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
            if (q & 1) mma_commit(empty(slot));
          }
          mma_commit(p_free);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
    const uint32_t done = warp < kPvWarp ? qk_done : o_full;
    if (elect_one()) mma_commit(done);
    __syncwarp();
    volatile int never = 0;
    mbar_wait(done, 0, &never);  // this warp's MMAs have finished before TMEM is read or freed
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // As in sga_attend.cu: thread t of the warp holds rows t/4 and 8 + t/4 of its
    // lane quarter, columns 8k + 2(t%4) and 8k + 2(t%4) + 1 for k = 0..7.
    const int quarter = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const int m4 = lane & 3;
    const int hrow[2] = {quarter * 16 + (lane >> 2), quarter * 16 + 8 + (lane >> 2)};  // this thread's two heads
    const uint32_t p_row = p_s + (2 * quarter + ((lane >> 3) & 1)) * 1024 + (lane & 7) * 128;  // stmatrix row
    float m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    // Every softmax thread runs every iteration, even after a wait ran out
    // (the abort flag then makes each later wait return at once), so the
    // named barriers below always see all 128 threads.
    {
      // Q: this warp's eight of the heads 32-63
      QPart v[2];
      const int head = 32 + 8 * (warp - kSoftmaxWarp) + (lane >> 3);
#pragma unroll
      for (int i = 0; i < 2; ++i) load_q(v[i], p.q, row, head + 4 * i, lane & 7);
#pragma unroll
      for (int i = 0; i < 2; ++i) store_q(v[i], q_s, q_scale, head + 4 * i, lane & 7, p.scale_log2);
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    bool ok = mbar_wait_warp(q_full, 0, abort_flag);
    const float sc[2] = {ok ? q_scale[hrow[0]] : 0.f, ok ? q_scale[hrow[1]] : 0.f};
    for (int j = 0; j < nchunks; ++j) {
      const int sb = j & 1;
      ok = ok && mbar_wait_warp(s_full(sb), static_cast<uint32_t>((j >> 1) & 1), abort_flag);
      tc_fence_after();
      float r[32];
      tmem_ld_16x256b_x8(tmem + lane_addr + kSCol + sb * kChunk, r);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(sb));
      // r[4k + 2i + e] = q.c of row i at column 8k + 2 m4 + e; masked slots -> -inf
      const uint64_t mk = *reinterpret_cast<volatile uint64_t*>(masks + j % kMaskRing);
      if (mk != ~0ull) {
        const uint64_t mine = mk >> (2 * m4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!((mine >> (8 * k + e)) & 1ull)) r[4 * k + e] = r[4 * k + 2 + e] = -INFINITY;
          }
        }
      }
      // The weights are computed with the running maximum so far, and again if this chunk passes it by more than the
      // threshold (or is the first).
      float mt[2], ps[2];
      uint32_t x[16];  // x[2k + i]: the weights of head i at columns 8k + 2 m4 and 8k + 2 m4 + 1
      bool need = false;
      const auto weights = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // every slot so far empty: -inf - 0, all weights zero
          const float m_p = m_ref[i] == -INFINITY ? 0.f : m_ref[i] - kPShift;
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          const bool exact = fabsf(m_p) < 0x1p20f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float v0 = r[4 * k + 2 * i], v1 = r[4 * k + 2 * i + 1];
            if (exact) {
              fma2(v0, v1, sc[i], -m_p);
            } else {  // scaled first and rounded, so that the maximum's difference is exact however large the scores are
              v0 = __fsub_rn(__fmul_rn(v0, sc[i]), m_p);
              v1 = __fsub_rn(__fmul_rn(v1, sc[i]), m_p);
            }
            v0 = fast_exp2(v0);
            v1 = fast_exp2(v1);
            x[2 * k + i] = pack_f16(v0, v1);
            add2(s[2 * (k & 1)], s[2 * (k & 1) + 1], v0, v1);
          }
          ps[i] = (s[0] + s[1]) + (s[2] + s[3]);
        }
      };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mp[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mp[c] = fmaxf(fmaxf(r[8 * c + 2 * i], r[8 * c + 2 * i + 1]), fmaxf(r[8 * c + 4 + 2 * i], r[8 * c + 5 + 2 * i]));
        mt[i] = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3]));
      }
      weights();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xFFFFFFFFu, mt[i], 1));
        mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xFFFFFFFFu, mt[i], 2)) * sc[i];  // the scale is positive
        need |= !(mt[i] <= m_ref[i] + kRescaleThreshold);                       // also for a NaN
      }
      // PV_{j-1} must be done before P and O are touched.
      ok = ok && mbar_wait_warp(p_free, static_cast<uint32_t>(j & 1) ^ 1u, abort_flag);
      tc_fence_after();
      if (named_barrier_or(1, kSoftmaxThreads, need)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float alpha = 1.f;
          if (m_ref[i] == -INFINITY) {
            m_ref[i] = mt[i];  // nothing accumulated yet (all earlier weights were zero)
          } else if (mt[i] > m_ref[i] + kRescaleThreshold) {
            alpha = exp2f(m_ref[i] - mt[i]);
            m_ref[i] = mt[i];
          }
          l_run[i] *= alpha;
          if (m4 == 0) head_f[hrow[i]] = alpha;
        }
        weights();
        if (j > 0) {
          named_barrier(1, kSoftmaxThreads);
          // O^T[dim][head] *= alpha[head], 32 heads of a block at a time: every lane holds one dim of each block.  Not
          // unrolled, or the registers that takes are spilled elsewhere.
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[32];
            const uint32_t src = tmem + lane_addr + c * 32;
            const float* f = head_f + (c & 1) * 32;
            tmem_ld32(src, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f[i];
            tmem_st32(src, o);
          }
          named_barrier(1, kSoftmaxThreads);
        }
      }
      l_run[0] += ps[0];  // this thread's columns
      l_run[1] += ps[1];
      // P[head][row] in the 128-byte-swizzled K-major layout (8 heads per 1 KB atom).  A thread's values are two
      // columns of row t/4 of 8 x 8 blocks, the layout stmatrix takes: four blocks (two of heads, two of columns)
      // at a time, the row addresses from lanes 8 b .. 8 b + 7 for block b.
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        stmatrix_x4(p_row + (((k + (lane >> 4)) ^ (lane & 7)) << 4), x[2 * k], x[2 * k + 1], x[2 * k + 2], x[2 * k + 3]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);  // P_j and any rescale of O
    }
    ok = ok && mbar_wait_warp(o_full, 0, abort_flag);
    if (!ok) {
      record_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l_run[i] += __shfl_xor_sync(0xFFFFFFFFu, l_run[i], 1);
      l_run[i] += __shfl_xor_sync(0xFFFFFFFFu, l_run[i], 2);
    }
    if (m4 == 0) {
      own_ml[hrow[0]] = make_float2(m_ref[0], l_run[0]);
      own_ml[hrow[1]] = make_float2(m_ref[1], l_run[1]);
    }
  }

  // ---- split merge: out = g / L * sum_r 2^(m_r - M) O_r with M = max_r m_r and L = sum_r 2^(m_r - M) l_r (per head).
  // Every thread of the cluster takes part in its barriers, on every path.
  const int S = p.splits;
  float* recv = reinterpret_cast<float*>(smem);          // value ring + rope slots + Q buffer, idle after the MMAs
  float* weight = reinterpret_cast<float*>(p_ptr);       // [S][64] the splits' factors, over P
  // One thread a head works out the factors: in a cluster one of the issuing warps, while the others send.
  const int head = warp * 32 + lane - kQkWarp * 32;
  const bool weighs = warp >= kQkWarp && warp < kQkWarp + 2;
  float g = 1.f;
  if (weighs && p.gate) g = sigmoidf_(bf16_bits_to_float(p.gate[static_cast<size_t>(row) * kHeads + head]));
  if (S > 1) {
    cluster.sync();  // every split's (m, l) published; all MMAs of every CTA done
    if (weighs) {
      // every split's (m, l) for this head, all loads in flight at once
      float2 ml[kMaxSplits];
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        ml[r] = r < S ? *cluster.map_shared_rank(&own_ml[head], r) : make_float2(-INFINITY, 0.f);
      float mx = -INFINITY;
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r) mx = fmaxf(mx, ml[r].x);
      float L = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r) {
        ml[r].x = ml[r].x == -INFINITY ? 0.f : exp2f(ml[r].x - mx);
        L += ml[r].x * ml[r].y;
      }
      const float f = L == 0.f ? 0.f : g / L;
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        if (r < S) weight[r * kHeads + head] = ml[r].x * f;
    }
  } else {
    __syncthreads();
    if (weighs) {
      const float l = own_ml[head].y;
      weight[head] = l == 0.f ? 0.f : g / l;
    }
    __syncthreads();
  }
  // With several splits, CTA r owns the float4 columns [v0(r), v0(r+1)) of
  // every head's 512 dims, v0(r) = 128 r / S; every CTA pushes its O for
  // those dims into the owner's receive buffer [source split][head][kStride].
  const int kStride = 4 * ((kDv / 4 + S - 1) / S);  // floats per (source, head) row: the widest slice
  if (warp < kProducerWarps || warp >= kSoftmaxWarp) {
    // Twelve warps read O^T out of TMEM: warp w reads lane quarter w % 4; the
    // producer warps 0-3 take dim block 0, 4-7 block 1, the softmax warps blocks 2-3.
    // O^T block b: this lane holds dim 128 b + 32 quarter + lane for all 64 heads.
    const int quarter = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const int blk0 = warp < 4 ? 0 : warp < kProducerWarps ? 1 : 2;
    const int blk1 = warp < kProducerWarps ? blk0 + 1 : 4;
    tc_fence_after();
    for (int c = 0; c < 2; ++c) {
      float f[32];  // the unsplit query's factors
      if (S == 1) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(f + i) = *reinterpret_cast<const float4*>(weight + c * 32 + i);
      }
      for (int blk = blk0; blk < blk1; ++blk) {
        const int dim = 128 * blk + 32 * quarter + lane;
        float o[32];
        tmem_ld32(tmem + lane_addr + blk * kHeads + c * 32, o);
        if (S == 1) {
          // neighbouring lanes trade a head: the even one stores both dims of head i, the odd one of head i + 1
          uint16_t* col = p.out + static_cast<size_t>(row) * kHeads * kDv +
                          static_cast<size_t>(c * 32 + (lane & 1)) * kDv + (dim & ~1);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float a = o[i] * f[i], b = o[i + 1] * f[i + 1];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? a : b, 1);
            *reinterpret_cast<uint32_t*>(col + static_cast<size_t>(i) * kDv) =
                lane & 1 ? pack_bf16(got, b) : pack_bf16(a, got);
          }
        } else {
          const int v = dim >> 2;
          const int owner = ((v + 1) * S - 1) / (kDv / 4);  // the r with v0(r) <= v < v0(r + 1)
          const int dl = dim - 4 * ((kDv / 4) * owner / S);
          SGA_DCHECK(p.status, owner < S && dl >= 0 && dl < kStride);
          float* col = cluster.map_shared_rank(recv + (split * kHeads + c * 32) * kStride + dl, owner);
#pragma unroll
          for (int i = 0; i < 32; ++i) col[i * kStride] = o[i];
        }
      }
    }
  }
  if (S > 1) {
    cluster.sync();  // every split's O delivered to its owners, and the weights written
    const int v0 = (kDv / 4) * split / S, v1 = (kDv / 4) * (split + 1) / S;
    const int vecs = v1 - v0;
    uint16_t* orow = p.out + static_cast<size_t>(row) * kHeads * kDv;
    for (int e = threadIdx.x; e < kHeads * vecs; e += kThreads) {
      const int h = e / vecs, dv = e - h * vecs;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r = 0; r < S; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(recv + (r * kHeads + h) * kStride + 4 * dv);
        const float f = weight[r * kHeads + h];
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
      *reinterpret_cast<uint2*>(orow + h * kDv + 4 * (v0 + dv)) =
          make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Splits of the K slots of each of `rows` queries: what a wave of clusters takes, in microseconds, times their number.
// Measured at 1 to 8 splits of 2,048 and 512 slots: 6.7 us beside the chunks, 1.3 us a chunk, and a merge of 3.6 us (4.6
// where the splits do not divide the dims evenly).  16 queries of 2,048 slots: 48.9 us unsplit, 21.8 in four, 21.1 in six,
// and in eight, which are more clusters than run at once, 31.8.
int attend4_splits(int rows, int chunks) {
  int best = 1;
  float best_us = 0.f;
  for (int s = 1; s <= chunks && s <= kMaxSplits; ++s) {
    const int waves = (rows + host::kClusters[s - 1] - 1) / host::kClusters[s - 1];
    const float merge = s == 1 ? 0.f : (s & (s - 1)) == 0 ? 3.6f : 4.6f;
    const float us = static_cast<float>(waves) * (6.7f + 1.31f * static_cast<float>((chunks + s - 1) / s) + merge);
    if (s == 1 || us < best_us) {
      best = s;
      best_us = us;
    }
  }
  return best;
}

cudaError_t launch_rows(Attend4Params p, int row0, int rows, int splits, cudaStream_t stream) {
  p.row0 = row0;
  p.splits = splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sga_attend4_kernel, p);
}

}  // namespace

cudaError_t launch_attend4(const Attend4Args& a, cudaStream_t stream) {
  const int rows = a.batch * a.n_q;
  cudaError_t e = cudaFuncSetAttribute(sga_attend4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  Attend4Params p;
  p.q = a.q;
  p.kv4 = a.kv4;
  p.idx = a.idx;
  p.gate = a.gate;
  p.out = a.out;
  p.status = a.status;
  p.n_q = a.n_q;
  p.kv_stride = a.kv_stride;
  p.top_k = a.top_k;
  p.chunks = a.top_k / kChunk;
  p.scale_log2 = static_cast<float>(SGA_SOFTMAX_SCALE * 1.4426950408889634);
  // Full waves of whole queries, then the rest with its slots split over the SMs it would leave idle: 512 queries of
  // 2,048 slots (3.46 waves) 198 us against 215 in one launch.
  const int tail = rows % host::kClusters[0];
  const int tail_splits = tail ? attend4_splits(tail, p.chunks) : 1;
  const int whole = tail_splits > 1 ? rows - tail : rows;
  if (whole > 0 && (e = launch_rows(p, 0, whole, 1, stream)) != cudaSuccess) return e;
  return whole < rows ? launch_rows(p, whole, tail, tail_splits, stream) : cudaSuccess;
}

}  // namespace sga
