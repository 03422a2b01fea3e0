// Quantisation along the rows, the operands of the 8-bit weight gradient: in every group, blocks of
// 128 rows of a column counted from the group's first row,
//
//   a = largest |x| of the block,  scale = a / 448 (at least 2^-126; 1 for zeros; NaN where the
//   block holds a NaN or an infinity),  q = e4m3(x / scale)
//
// the blockwise rule of quant.cuh turned by 90 degrees.  Rows may be gathered: row r of q comes
// from the token whose slot lies in row r.  Bound by HBM: each element is read once, kept in
// registers while its block's largest magnitude is found, and written once.
//
// A block of threads takes 128 rows x 128 columns: thread (i, c) the 8 columns 8 c.. of the rows
// i, i + 16, .., so that 16 threads read 256 bytes of a row (16-bit) and write 128.  Which rows
// those are the offsets say: block b of the scales belongs to the last group e with
// offsets[e] / 128 + e <= b, which the threads count together.
#include <cuda_fp16.h>

#include "expert_ops.cuh"
#include "moe_ops.cuh"
#include "quant.cuh"

namespace bsfp8 {
namespace {

constexpr int kBlockRows = 128, kTileCols = 128;
constexpr int kThreads = 256;
constexpr int kColumnThreads = kTileCols / 8;            // threads side by side
constexpr int kRowThreads = kThreads / kColumnThreads;   // 16
constexpr int kRowsEach = kBlockRows / kRowThreads;      // 8

template <int XT>
struct Eight {  // elements of a row, as they are stored
  uint32_t w[XT == E_FP32 ? 8 : 4];
};

template <int XT>
__device__ __forceinline__ void unpack(const Eight<XT>& r, float (&v)[8]) {
  if constexpr (XT == E_FP32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (XT == E_BF16) {
        unpack_bf16x2(r.w[j], v[2 * j], v[2 * j + 1]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  }
}

template <int XT, bool GATHER>
__global__ void __launch_bounds__(kThreads, XT == E_FP32 ? 2 : 4) columns_kernel(ColumnsArgs a) {
  __shared__ float part[kThreads / 32][kTileCols];
  const int b = blockIdx.x;
  // the groups whose first block is b or before it; a group's first block grows with the group
  int before = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) before += a.offsets[e] / kBlockRows + e <= b;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) before += __shfl_xor_sync(0xffffffffu, before, d);
  __shared__ int counts[kThreads / 32];
  if (threadIdx.x % 32 == 0) counts[threadIdx.x / 32] = before;
  __syncthreads();
  int e = -1;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) e += counts[i];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {
    int64_t unused;
    const int status = check_groups<1>(a.offsets, nullptr, a.E, a.E, a.M_total, unused);
    if (status && threadIdx.x == 0) atomicCAS(a.err, 0, status);
  }
  if (e < 0) return;
  const int64_t r0 = a.offsets[e], r1 = a.offsets[e + 1];
  const int64_t first = r0 + (b - (r0 / kBlockRows + e)) * (int64_t)kBlockRows;
  // a block that no group has, or offsets that are no partition (recorded above)
  if (r0 < 0 || r1 > a.M_total || first < r0 || first >= r1) return;
  const int rows = r1 - first < kBlockRows ? (int)(r1 - first) : kBlockRows;

  const int c = threadIdx.x % kColumnThreads, i0 = threadIdx.x / kColumnThreads;
  const int col = blockIdx.y * kTileCols + 8 * c;
  constexpr int kBytes = XT == E_FP32 ? 4 : 2;
  int64_t from[kRowsEach];
#pragma unroll
  for (int j = 0; j < kRowsEach; ++j) {
    const int i = i0 + j * kRowThreads;
    from[j] = -1;
    if (i < rows) {
      if constexpr (GATHER) {
        const int slot = a.slot_of_row[first + i];
        from[j] = slot < 0 ? -1 : slot / a.top_k;
      } else {
        from[j] = first + i;
      }
    }
  }
  Eight<XT> x[kRowsEach];
#pragma unroll
  for (int j = 0; j < kRowsEach; ++j) {
    if constexpr (GATHER) {
      if (from[j] >= a.x_rows) {
        atomicCAS(a.err, 0, DEV_BAD_ROWS);
        from[j] = -1;
      }
    }
#pragma unroll
    for (uint32_t& w : x[j].w) w = 0;
    if (from[j] >= 0)
      load_words<sizeof(Eight<XT>) / 4>(
          static_cast<const char*>(a.x) + (from[j] * a.K + col) * kBytes, x[j].w);
  }
  float top[8] = {};
#pragma unroll
  for (int j = 0; j < kRowsEach; j += 2) {
    float v[8], u[8];
    unpack<XT>(x[j], v);
    unpack<XT>(x[j + 1], u);
#pragma unroll
    for (int k = 0; k < 8; ++k) top[k] = max3_nan(top[k], fabsf(v[k]), fabsf(u[k]));
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) top[k] = max_nan(top[k], __shfl_xor_sync(0xffffffffu, top[k], 16));
  if (threadIdx.x % 32 < kColumnThreads) {
    float4* p = reinterpret_cast<float4*>(&part[threadIdx.x / 32][8 * c]);
    p[0] = make_float4(top[0], top[1], top[2], top[3]);
    p[1] = make_float4(top[4], top[5], top[6], top[7]);
  }
  __syncthreads();
  if (threadIdx.x < kTileCols) {  // one column each: its scale, and the scale's reciprocal
    float m = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) m = max_nan(m, part[w][threadIdx.x]);
    const bool finite = m < __int_as_float(0x7f800000);
    const float scale = m == 0.0f ? 1.0f : fmaxf(__fdiv_rn(m, 448.0f), 0x1p-126f);
    a.scales[(int64_t)b * a.K + blockIdx.y * kTileCols + threadIdx.x] =
        finite ? scale : __int_as_float(0x7fffffff);
    part[0][threadIdx.x] = finite ? __frcp_rn(scale) : 0.0f;
  }
  __syncthreads();
  float inv[8];
  {
    const float4* p = reinterpret_cast<const float4*>(&part[0][8 * c]);
    const float4 lo = p[0], hi = p[1];
    inv[0] = lo.x; inv[1] = lo.y; inv[2] = lo.z; inv[3] = lo.w;
    inv[4] = hi.x; inv[5] = hi.y; inv[6] = hi.z; inv[7] = hi.w;
  }
#pragma unroll
  for (int j = 0; j < kRowsEach; ++j) {
    const int i = i0 + j * kRowThreads;
    if (i >= rows) break;
    float v[8];
    unpack<XT>(x[j], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= inv[k];
    const uint32_t lo = cvt_e4m3x2(v[0], v[1]) | (cvt_e4m3x2(v[2], v[3]) << 16);
    const uint32_t hi = cvt_e4m3x2(v[4], v[5]) | (cvt_e4m3x2(v[6], v[7]) << 16);
    *reinterpret_cast<uint2*>(a.q + (first + i) * a.K + col) = make_uint2(lo, hi);
  }
}

template <int XT>
cudaError_t columns_as(const ColumnsArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(a.M_total / kBlockRows + a.E), (unsigned)(a.K / kTileCols));
  if (a.slot_of_row) columns_kernel<XT, true><<<grid, kThreads, 0, stream>>>(a);
  else columns_kernel<XT, false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_columns(int x_type, const ColumnsArgs& a, cudaStream_t stream) {
  switch (x_type) {
    case E_BF16: return columns_as<E_BF16>(a, stream);
    case E_FP16: return columns_as<E_FP16>(a, stream);
    default: return columns_as<E_FP32>(a, stream);
  }
}

}  // namespace bsfp8
