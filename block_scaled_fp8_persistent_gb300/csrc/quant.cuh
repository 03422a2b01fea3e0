// Block quantisation of a row's values, shared by the operators that write GEMM operands
// (moe_quant.cu).  A thread holds 16 consecutive elements of a row in fp32; the 1, 2 or 8
// neighbouring threads that share a scale block agree on its largest magnitude with shuffles.
//
//   format      elements   scale                         block   largest value
//   mxfp8       e4m3       UE8M0, 2^ceil(log2(a/448))    32      448
//   mxfp4       e2m1       UE8M0, 2^ceil(log2(a/6))      32      6
//   nvfp4       e2m1       e4m3(a/6), at least 2^-9      16      6
//   blockwise   e4m3       fp32, a/448                   128     448
//
// a is the block's largest magnitude; an all-zero block has scale 1, a block that holds a NaN
// or an infinity a NaN scale, so that whatever is computed of it is NaN.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "ptx.cuh"

namespace bsfp8 {

enum QuantFormat : int { Q_MXFP8 = 0, Q_MXFP4 = 1, Q_NVFP4 = 2, Q_BLOCKWISE = 3 };

template <int FMT>
struct QuantTraits {
  static constexpr bool fp4 = FMT == Q_MXFP4 || FMT == Q_NVFP4;
  static constexpr int vec = FMT == Q_BLOCKWISE ? 128 : FMT == Q_NVFP4 ? 16 : 32;
  static constexpr int group = vec / 16;      // threads per scale block
  static constexpr int words = fp4 ? 2 : 4;   // 32-bit words of codes per thread
};

// Two products at once.
__device__ __forceinline__ void mul2(float a0, float a1, float b0, float b1, float& r0, float& r1) {
  asm("{\n\t.reg .b64 a, b, r;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two values to e4m3, lo in the low byte: round to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight values to e2m1, element i in nibble i: round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// A thread's 16 quantised elements and its block's scale (UE8M0 or e4m3 code, or fp32 bits).
template <int FMT>
struct Quantised {
  uint32_t w[QuantTraits<FMT>::words];
  uint32_t scale;
};

// Every lane of a warp calls this together; the threads of one scale block are neighbours.
template <int FMT>
__device__ __forceinline__ Quantised<FMT> quantise16(const float (&v)[16]) {
  using T = QuantTraits<FMT>;
  float a = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 15; i += 2) a = max3_nan(a, fabsf(v[i]), fabsf(v[i + 1]));
  a = max_nan(a, fabsf(v[15]));
#pragma unroll
  for (int d = 1; d < T::group; d *= 2) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, d));

  Quantised<FMT> out;
  const bool finite = a < __int_as_float(0x7f800000);
  float inv, scale = 1.0f;
  if constexpr (FMT == Q_MXFP8 || FMT == Q_MXFP4) {
    // a = m * 2^x with 1 <= m < 2: ceil(log2(a / 448)) = x - 8 + (m > 1.75), and
    // ceil(log2(a / 6)) = x - 2 + (m > 1.5), on the exponent field as it is
    const uint32_t bits = __float_as_uint(a);
    const int lead = T::fp4 ? 0x400000 : 0x600000;
    int code = (int)(bits >> 23) - (T::fp4 ? 2 : 8) + ((int)(bits & 0x7fffff) > lead ? 1 : 0);
    code = a == 0.0f ? 127 : code < 0 ? 0 : code;
    inv = __uint_as_float((uint32_t)(254 - code) << 23);  // 2^(127 - code): exact
    out.scale = finite ? (uint32_t)code : 255u;
  } else if constexpr (FMT == Q_NVFP4) {
    const float s = fminf(fmaxf(__fdiv_rn(a, 6.0f), 0.001953125f), 448.0f);
    const uint32_t code = a == 0.0f ? 0x38u : cvt_e4m3x2(s, 0.0f);
    // the code's value: exponent and fraction moved into place, times 2^120 for the biases
    scale = __uint_as_float((code & 0x7f) << 20) * 0x1p120f;
    inv = __frcp_rn(scale);
    out.scale = finite ? code : 0x7fu;
  } else {
    scale = a == 0.0f ? 1.0f : fmaxf(__fdiv_rn(a, 448.0f), 0x1p-126f);
    inv = __frcp_rn(scale);
    out.scale = finite ? __float_as_uint(scale) : 0x7fffffffu;
  }
  if (!finite) inv = 0.0f;

  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = v[i] * inv;
    // A bf16 value over an e4m3 scale is often exactly half way between two e2m1 values, and
    // the rounded reciprocal can miss it: one Newton step on the quotient gives v / scale
    // correctly rounded, so that ties go to even.
    if constexpr (FMT == Q_NVFP4) y[i] = __fmaf_rn(__fmaf_rn(-y[i], scale, v[i]), inv, y[i]);
  }
  if constexpr (T::fp4) {
    out.w[0] = cvt_e2m1x8(y);
    out.w[1] = cvt_e2m1x8(y + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      out.w[i] = cvt_e4m3x2(y[4 * i], y[4 * i + 1]) | (cvt_e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16);
  }
  return out;
}

// Stores the thread's codes of elements 16 * item .. of row `row` of an operand of K columns.
template <int FMT>
__device__ __forceinline__ void store_codes(const Quantised<FMT>& o, uint8_t* q, int64_t row,
                                            int item, int K) {
  if constexpr (QuantTraits<FMT>::fp4)
    *reinterpret_cast<uint2*>(q + row * (K / 2) + item * 8) = make_uint2(o.w[0], o.w[1]);
  else
    *reinterpret_cast<uint4*>(q + row * K + (int64_t)item * 16) =
        make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
}

// Stores the block's scale, from the first of its threads; the operand has `rows` rows.
template <int FMT>
__device__ __forceinline__ void store_scale(const Quantised<FMT>& o, void* scales, int64_t row,
                                            int64_t rows, int item, int K) {
  using T = QuantTraits<FMT>;
  if (item % T::group != 0) return;
  if constexpr (FMT == Q_BLOCKWISE) {
    // Rows next to each other fill a sector from several blocks: it is to stay in L2 until they
    // have, or it goes to memory in parts (8192 rows of 7168 to 8 places with their sort 98.7 us
    // at the default priority, 92.7 so, 86.9 without any scales).
    asm volatile("st.global.L2::cache_hint.b32 [%0], %1, %2;" ::"l"(
                     static_cast<uint32_t*>(scales) + (item / T::group) * rows + row),
                 "r"(o.scale), "l"(l2_policy_evict_last())
                 : "memory");
  } else {
    static_cast<uint8_t*>(scales)[row * (K / T::vec) + item / T::group] = (uint8_t)o.scale;
  }
}

__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}

// WORDS 32-bit words from p, 16-byte aligned, or 32-byte aligned where WIDE.  Not the read-only
// path: a caller may pass the norm's residual as its output too.
template <int WORDS, bool WIDE = false>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[WORDS]) {
  const char* c = static_cast<const char*>(p);
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 8)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]),
                     "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(c + 4 * i));
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "l"(c + 4 * i));
  }
}

}  // namespace bsfp8
