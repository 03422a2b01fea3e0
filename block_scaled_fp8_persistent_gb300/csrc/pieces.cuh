// 16-element pieces of a row, as the element-wise operators read them (moe_quant.cu,
// swiglu_grad.cu), and the approximate instructions of SwiGLU.
#pragma once
#include <cuda_fp16.h>
#include <cstdint>

#include "moe_ops.cuh"
#include "quant.cuh"

namespace bsfp8 {

// 16 elements as they are stored, and as fp32.
template <int XT>
constexpr int kWords = XT == E_FP32 ? 16 : 8;

template <int XT>
__device__ __forceinline__ void to_float(const uint32_t (&w)[kWords<XT>], float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < kWords<XT>; ++i) {
    if constexpr (XT == E_FP32) {
      v[i] = __uint_as_float(w[i]);
    } else if constexpr (XT == E_BF16) {
      unpack_bf16x2(w[i], v[2 * i], v[2 * i + 1]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <int XT, bool WIDE = false>
__device__ __forceinline__ void load16(const void* x, int64_t at, float (&v)[16]) {
  uint32_t w[kWords<XT>];
  load_words<kWords<XT>, WIDE>(static_cast<const char*>(x) + at * (XT == E_FP32 ? 4 : 2), w);
  to_float<XT>(w, v);
}

// 1 / x for x >= 1, within an ulp; 0 where it would be subnormal.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace bsfp8
