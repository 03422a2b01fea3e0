// Operators that write a grouped GEMM's operand: quantisation of rows (in place, or sorted by
// expert), RMS norm with the residual's addition, SwiGLU.  All are bound by HBM: each element
// is read once, its block quantised in registers (quant.cuh) and written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "moe_ops.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace bsfp8 {
namespace {

bool wide(const void* p) { return (reinterpret_cast<uintptr_t>(p) % 32) == 0; }

template <int XT, bool WIDE>
__device__ __forceinline__ void load16(const void* x, int64_t at, float (&v)[16]) {
  if constexpr (XT == E_FP32) {
    uint32_t w[16];
    load_stream<16, WIDE>(static_cast<const float*>(x) + at, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
  } else {
    uint32_t w[8];
    load_stream<8, WIDE>(static_cast<const uint16_t*>(x) + at, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (XT == E_BF16) {
        unpack_bf16x2(w[i], v[2 * i], v[2 * i + 1]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// quantise rows; with a row map, each row goes to the rows its slots name
// ---------------------------------------------------------------------------------------
template <int FMT, int XT, bool WIDE, bool MAP>
__global__ void __launch_bounds__(512) quantize_kernel(QuantizeArgs a) {
  const int64_t t = blockIdx.x;
  const int items = a.K / 16;
  for (int i = threadIdx.x; i < (items + 31) / 32 * 32; i += blockDim.x) {
    float v[16] = {};
    if (i < items) load16<XT, WIDE>(a.x, t * a.K + (int64_t)i * 16, v);
    const Quantised<FMT> o = quantise16<FMT>(v);
    if (i >= items) continue;
    if constexpr (!MAP) {
      store_quantised<FMT>(o, a.q, a.scales, t, a.out_rows, i, a.K);
    } else {
      for (int j = 0; j < a.top_k; ++j) {
        const int row = __ldg(a.row_of_slot + t * a.top_k + j);
        if (row >= a.out_rows) atomicCAS(a.err, 0, DEV_BAD_ROWS);
        if (row >= 0 && row < a.out_rows)
          store_quantised<FMT>(o, a.q, a.scales, row, a.out_rows, i, a.K);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// RMS norm: h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight
// ---------------------------------------------------------------------------------------
template <int FMT, bool Q, int RT, int ITEMS, bool WIDE>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormArgs a) {
  __shared__ float part[32];
  const int64_t t = blockIdx.x;
  const int items = a.K / 16;
  float h[ITEMS][16];
  float sum = 0.0f;
#pragma unroll
  for (int n = 0; n < ITEMS; ++n) {
    const int i = threadIdx.x + n * blockDim.x;
#pragma unroll
    for (int e = 0; e < 16; ++e) h[n][e] = 0.0f;
    if (i < items) {
      const int64_t at = t * a.K + (int64_t)i * 16;
      load16<E_BF16, WIDE>(a.x, at, h[n]);
      if (a.residual) {
        float r[16];
        load16<RT, WIDE>(a.residual, at, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) h[n][e] += r[e];
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) sum = fmaf(h[n][e], h[n][e], sum);
      if (a.residual_out) {
        if constexpr (RT == E_FP32) {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.residual_out) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            d[e] = make_float4(h[n][4 * e], h[n][4 * e + 1], h[n][4 * e + 2], h[n][4 * e + 3]);
        } else {
          uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.residual_out) + at);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            d[e] = make_uint4(pack_bf16x2(h[n][8 * e], h[n][8 * e + 1]),
                              pack_bf16x2(h[n][8 * e + 2], h[n][8 * e + 3]),
                              pack_bf16x2(h[n][8 * e + 4], h[n][8 * e + 5]),
                              pack_bf16x2(h[n][8 * e + 6], h[n][8 * e + 7]));
        }
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  sum = threadIdx.x % 32 < blockDim.x / 32 ? part[threadIdx.x % 32] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float r = rsqrtf(sum / (float)a.K + a.eps);
#pragma unroll
  for (int n = 0; n < ITEMS; ++n) {
    const int i = threadIdx.x + n * blockDim.x;
    if (i < items) {
      const uint4* wp =
          reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + i * 16);
      const uint4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
      const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float lo, hi;
        unpack_bf16x2(w[e], lo, hi);
        h[n][2 * e] *= r * lo;
        h[n][2 * e + 1] *= r * hi;
      }
      if (a.y) {
        uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + t * a.K + (int64_t)i * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          d[e] = make_uint4(pack_bf16x2(h[n][8 * e], h[n][8 * e + 1]),
                            pack_bf16x2(h[n][8 * e + 2], h[n][8 * e + 3]),
                            pack_bf16x2(h[n][8 * e + 4], h[n][8 * e + 5]),
                            pack_bf16x2(h[n][8 * e + 6], h[n][8 * e + 7]));
      }
    }
    if constexpr (Q) {
      const Quantised<FMT> o = quantise16<FMT>(h[n]);
      if (i < items) store_quantised<FMT>(o, a.q, a.scales, t, a.rows, i, a.K);
    }
  }
}

// ---------------------------------------------------------------------------------------
// SwiGLU: g / (1 + exp(-g)) * u
// ---------------------------------------------------------------------------------------
template <int FMT, bool WIDE>
__global__ void __launch_bounds__(512) swiglu_kernel(SwigluArgs a) {
  const int64_t t = blockIdx.x;
  const int items = a.N / 16;
  for (int i = threadIdx.x; i < (items + 31) / 32 * 32; i += blockDim.x) {
    float v[16] = {};
    if (i < items) {
      float u[16];
      const int64_t at = t * 2 * a.N + (int64_t)i * 16;
      load16<E_BF16, WIDE>(a.h, at, v);
      load16<E_BF16, WIDE>(a.h, at + a.N, u);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = __fdividef(v[e], 1.0f + __expf(-v[e])) * u[e];
    }
    const Quantised<FMT> o = quantise16<FMT>(v);
    if (i < items) store_quantised<FMT>(o, a.q, a.scales, t, a.rows, i, a.N);
  }
}

int block_for(int items, int most) {
  const int t = (items + 31) / 32 * 32;
  return t < most ? t : most;
}

template <int FMT, int XT, bool WIDE>
cudaError_t quantize_as(const QuantizeArgs& a, cudaStream_t stream) {
  const int threads = block_for(a.K / 16, 512);
  if (a.row_of_slot)
    quantize_kernel<FMT, XT, WIDE, true><<<(unsigned)a.rows, threads, 0, stream>>>(a);
  else
    quantize_kernel<FMT, XT, WIDE, false><<<(unsigned)a.rows, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t quantize_format(int x_type, const QuantizeArgs& a, cudaStream_t stream) {
  const bool w = wide(a.x);
  switch (x_type) {
    case E_BF16: return w ? quantize_as<FMT, E_BF16, true>(a, stream) : quantize_as<FMT, E_BF16, false>(a, stream);
    case E_FP16: return w ? quantize_as<FMT, E_FP16, true>(a, stream) : quantize_as<FMT, E_FP16, false>(a, stream);
    default: return w ? quantize_as<FMT, E_FP32, true>(a, stream) : quantize_as<FMT, E_FP32, false>(a, stream);
  }
}

template <int FMT, bool Q, int RT, bool WIDE>
cudaError_t norm_as(const NormArgs& a, cudaStream_t stream) {
  const int items = a.K / 16;
  if (items <= 1024)
    rmsnorm_kernel<FMT, Q, RT, 1, WIDE><<<(unsigned)a.rows, block_for(items, 1024), 0, stream>>>(a);
  else
    rmsnorm_kernel<FMT, Q, RT, 2, WIDE><<<(unsigned)a.rows, block_for((items + 1) / 2, 1024), 0, stream>>>(a);
  return cudaGetLastError();
}

template <int FMT, bool Q>
cudaError_t norm_format(int residual_type, const NormArgs& a, cudaStream_t stream) {
  const bool w = wide(a.x) && wide(a.residual);
  if (residual_type == E_FP32)
    return w ? norm_as<FMT, Q, E_FP32, true>(a, stream) : norm_as<FMT, Q, E_FP32, false>(a, stream);
  return w ? norm_as<FMT, Q, E_BF16, true>(a, stream) : norm_as<FMT, Q, E_BF16, false>(a, stream);
}

template <int FMT>
cudaError_t swiglu_format(const SwigluArgs& a, cudaStream_t stream) {
  const int threads = block_for(a.N / 16, 512);
  if (wide(a.h))
    swiglu_kernel<FMT, true><<<(unsigned)a.rows, threads, 0, stream>>>(a);
  else
    swiglu_kernel<FMT, false><<<(unsigned)a.rows, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(int format, int x_type, const QuantizeArgs& a, cudaStream_t stream) {
  switch (format) {
    case Q_MXFP8: return quantize_format<Q_MXFP8>(x_type, a, stream);
    case Q_MXFP4: return quantize_format<Q_MXFP4>(x_type, a, stream);
    case Q_NVFP4: return quantize_format<Q_NVFP4>(x_type, a, stream);
    default: return quantize_format<Q_BLOCKWISE>(x_type, a, stream);
  }
}

cudaError_t launch_rmsnorm_quant(int format, int residual_type, const NormArgs& a,
                                 cudaStream_t stream) {
  if (!a.q) return norm_format<Q_MXFP8, false>(residual_type, a, stream);
  switch (format) {
    case Q_MXFP8: return norm_format<Q_MXFP8, true>(residual_type, a, stream);
    case Q_MXFP4: return norm_format<Q_MXFP4, true>(residual_type, a, stream);
    case Q_NVFP4: return norm_format<Q_NVFP4, true>(residual_type, a, stream);
    default: return norm_format<Q_BLOCKWISE, true>(residual_type, a, stream);
  }
}

cudaError_t launch_swiglu_quant(int format, const SwigluArgs& a, cudaStream_t stream) {
  switch (format) {
    case Q_MXFP8: return swiglu_format<Q_MXFP8>(a, stream);
    case Q_MXFP4: return swiglu_format<Q_MXFP4>(a, stream);
    case Q_NVFP4: return swiglu_format<Q_NVFP4>(a, stream);
    default: return swiglu_format<Q_BLOCKWISE>(a, stream);
  }
}

}  // namespace bsfp8
