// The 4-bit latent cache: its writer and reader, and the C-ABI calls over it
// (the attention kernel is in sga_attend4.cu).  Row layout in sga.h.
//
// Both kernels give a row to one warp: a lane owns one group of 16 latent dims
// (32 bytes of bf16, 8 bytes of codes, one scale) and two rope values, so a row
// needs no exchange between lanes and every access is a whole row of
// consecutive lanes.  They are bound by the bytes they move (1,152 in and 416
// out, or the reverse) and, for the few rows of a decode step, by the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sga.h"
#include "sga_host.h"
#include "sga_internal.cuh"
#include "sga_ptx.cuh"

namespace {

using sga::host::aligned;
using sga::host::at;

constexpr int kLatent = SGA_V_DIM;              // 512
constexpr int kKvDim = SGA_QK_DIM;              // 576
constexpr int kRowBytes = SGA_KV4_ROW_BYTES;    // 416
constexpr int kScaleOff = kLatent / 2;
constexpr int kRopeOff = kScaleOff + kLatent / 16;
constexpr int kWarps = 8;                       // rows per block

__global__ void __launch_bounds__(32 * kWarps) kv4_append_kernel(const uint16_t* kv_rows, const int32_t* q_pos,
                                                                 uint8_t* kv4, int* status, long long rows, int n_q,
                                                                 int kv_stride) {
  sga::grid_dependency_wait();
  sga::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int pos = __ldg(q_pos + row);
  if (pos < 0 || pos >= kv_stride) {
    if (lane == 0) sga::record_status(status, sga::kStatusDeviceArg);
    return;
  }
  const uint8_t* src = reinterpret_cast<const uint8_t*>(kv_rows) + row * (kKvDim * 2);
  uint8_t* dst = kv4 + (row / n_q * kv_stride + pos) * kRowBytes;
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(src + 32 * lane));
  const uint4 b = __ldg(reinterpret_cast<const uint4*>(src + 32 * lane + 16));
  const uint32_t rope = __ldg(reinterpret_cast<const uint32_t*>(src + 2 * kLatent + 4 * lane));
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float x[16], top = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    nan |= isnan(x[2 * i]) || isnan(x[2 * i + 1]);
  }
  // top / 6 and x / scale have at most 8 significant bits over at most 4, so a
  // quotient is either a rounding tie exactly or further from it than an fp32
  // step: rounding to fp32 first never changes the E4M3 or E2M1 result.
  const uint8_t scale = __nv_cvt_float_to_fp8(__fdiv_rn(top, 6.f), __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(scale, __NV_E4M3)));
  uint32_t codes[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = s > 0.f ? make_float2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s))
                             : make_float2(copysignf(0.f, x[2 * i]), copysignf(0.f, x[2 * i + 1]));
    codes[i >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest)) << (8 * (i & 3));
  }
  if (nan) codes[0] = codes[1] = 0;
  *reinterpret_cast<uint2*>(dst + 8 * lane) = make_uint2(codes[0], codes[1]);
  dst[kScaleOff + lane] = nan ? 0x7F : scale;
  *reinterpret_cast<uint32_t*>(dst + kRopeOff + 4 * lane) = rope;
}

__global__ void __launch_bounds__(32 * kWarps) kv4_read_kernel(const uint8_t* kv4, const int32_t* pos_in,
                                                               uint16_t* kv_rows, int* status, long long rows, int n_q,
                                                               int kv_stride) {
  sga::grid_dependency_wait();
  sga::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int pos = __ldg(pos_in + row);
  const bool valid = pos >= 0 && pos < kv_stride;
  if ((pos < -1 || pos >= kv_stride) && lane == 0) sga::record_status(status, sga::kStatusDeviceArg);
  uint2 codes = make_uint2(0, 0);
  uint8_t scale = 0;
  uint32_t rope = 0;
  if (valid) {
    const uint8_t* src = kv4 + (row / n_q * kv_stride + pos) * kRowBytes;
    codes = *reinterpret_cast<const uint2*>(src + 8 * lane);
    scale = src[kScaleOff + lane];
    rope = *reinterpret_cast<const uint32_t*>(src + kRopeOff + 4 * lane);
  }
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(scale, __NV_E4M3)));
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t byte = ((i < 4 ? codes.x : codes.y) >> (8 * (i & 3))) & 0xFFu;
    const float2 v = __half22float2(
        __half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1)));
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * s, v.y * s);  // at most 6 significant bits: exact
    o[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  uint8_t* dst = reinterpret_cast<uint8_t*>(kv_rows) + row * (kKvDim * 2);
  *reinterpret_cast<uint4*>(dst + 32 * lane) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(dst + 32 * lane + 16) = make_uint4(o[4], o[5], o[6], o[7]);
  *reinterpret_cast<uint32_t*>(dst + 2 * kLatent + 4 * lane) = rope;
}

// The sizes of a cache call (top_k plays no part in it).
bool cache_dims_ok(const sga_dims_t* d) {
  if (!d || d->batch < 1 || d->n_q < 1 || d->kv_stride < 1 || d->kv_stride > SGA_MAX_KV_STRIDE) return false;
  const long long rows = static_cast<long long>(d->batch) * d->n_q;
  return rows * 64 <= INT32_MAX && static_cast<long long>(d->batch) * d->kv_stride <= INT32_MAX;
}

bool attend_dims_ok(const sga_dims_t* d) {
  return cache_dims_ok(d) && d->top_k >= 64 && d->top_k <= SGA_MAX_TOP_K && d->top_k % 64 == 0;
}

bool ws_ok(const void* ws, size_t ws_bytes) {
  return aligned(ws, sga::host::kWsAlign) && ws_bytes >= sga::host::kStatusBytes;
}

}  // namespace

namespace sga {

cudaError_t launch_kv4_append(const uint16_t* kv_rows, const int32_t* q_pos, uint8_t* kv4, int* status, int batch,
                              int n_q, int kv_stride, cudaStream_t s) {
  const long long rows = static_cast<long long>(batch) * n_q;
  return host::launch_pdl(kv4_append_kernel, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)),
                          dim3(32 * kWarps), 0, s, kv_rows, q_pos, kv4, status, rows, n_q, kv_stride);
}

}  // namespace sga

extern "C" {

sga_status_t sga_kv4_append(const sga_dims_t* dims, const sga_bf16_t* kv_rows, const int32_t* q_pos, uint8_t* kv4,
                            void* ws, size_t ws_bytes, sga_stream_t stream) {
  if (!cache_dims_ok(dims)) return SGA_ERR_INVALID_ARG;
  if (!aligned(kv_rows, 16) || !aligned(q_pos, 4) || !aligned(kv4, 32)) return SGA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes)) return SGA_ERR_WORKSPACE;
  int sms = 0;
  const sga_status_t st = sga::host::device_info(&sms);
  if (st != SGA_OK) return st;
  sga::host::NvtxRange range("sga.kv4_append");
  return sga::host::from_cuda(sga::launch_kv4_append(kv_rows, q_pos, kv4, at<int>(ws, 0), dims->batch, dims->n_q,
                                                     dims->kv_stride, static_cast<cudaStream_t>(stream)));
}

sga_status_t sga_kv4_read(const sga_dims_t* dims, const uint8_t* kv4, const int32_t* pos, sga_bf16_t* kv_rows,
                          void* ws, size_t ws_bytes, sga_stream_t stream) {
  if (!cache_dims_ok(dims)) return SGA_ERR_INVALID_ARG;
  if (!aligned(kv_rows, 16) || !aligned(pos, 4) || !aligned(kv4, 32)) return SGA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes)) return SGA_ERR_WORKSPACE;
  int sms = 0;
  const sga_status_t st = sga::host::device_info(&sms);
  if (st != SGA_OK) return st;
  sga::host::NvtxRange range("sga.kv4_read");
  const long long rows = static_cast<long long>(dims->batch) * dims->n_q;
  return sga::host::from_cuda(sga::host::launch_pdl(
      kv4_read_kernel, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0,
      static_cast<cudaStream_t>(stream), kv4, pos, kv_rows, at<int>(ws, 0), rows, dims->n_q, dims->kv_stride));
}

sga_status_t sga_sparse_mla_attend_kv4(const sga_dims_t* dims, const sga_bf16_t* q, const uint8_t* kv4,
                                       const int32_t* idx, const sga_bf16_t* gate, sga_bf16_t* out, void* ws,
                                       size_t ws_bytes, sga_stream_t stream) {
  if (!attend_dims_ok(dims)) return SGA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv4, 32) || !aligned(idx, 16) || !aligned(out, 16) || (gate && !aligned(gate, 2)))
    return SGA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes)) return SGA_ERR_WORKSPACE;
  int sms = 0;
  const sga_status_t st = sga::host::device_info(&sms);
  if (st != SGA_OK) return st;
  sga::host::NvtxRange range("sga.sparse_mla_attend_kv4");
  sga::Attend4Args a{q, kv4, idx, gate, out, at<int>(ws, 0), dims->batch, dims->n_q, dims->kv_stride, dims->top_k};
  return sga::host::from_cuda(sga::launch_attend4(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
