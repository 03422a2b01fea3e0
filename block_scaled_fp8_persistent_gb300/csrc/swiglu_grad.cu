// SwiGLU's gradient: with s = 1 / (1 + exp(-g)) and act = g s u,
//
//   d_u = d g s,   d_g = d u s (1 + g (1 - s))
//
// written in 16 bits and / or quantised as the A of the products that follow, and act itself.  Bound
// by HBM: a thread reads 16 elements of each of g, u and d once and writes what is made of them (65536
// rows of 2048 with d_h, act and blockwise d_h: 297 us, 6.4 TB/s).  Straight pieces, no loop: three
// blocks of 256 threads to an SM hold their 48 values without spilling, and the rest is other blocks'.
#include "moe_ops.cuh"
#include "pieces.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace bsfp8 {
namespace {

constexpr int kPieceThreads = 256;

// s and 1 - s.  What is quantised is not rounded before, and blockwise scales are fp32: there (EXACT)
// exp(-g) is the library's, to 2 units, and 1 - s is exp(-g) s for g > 0, where the difference would
// lose |g| 2^-25 beside 1.  Else the exponential is the forward's, 2^t of a rounded t, off by |g| 2^-24,
// which goes whole into both gradients where g < 0: at most 5e-6, a hundredth of half a step of fp16
// and less of bf16 and of the codes of 8 and 4 bits.  65536 rows of 2048, exact and not: blockwise with
// d_h and act 297 us either way; d_h 220 and 212, mxfp8 223 and 210, act alone 148 and 132.
template <bool EXACT>
struct Sigmoid {
  float s, rest;
  __device__ __forceinline__ explicit Sigmoid(float g) {
    if constexpr (EXACT) {
      const float e = expf(-g);
      s = rcp_approx(1.0f + e);
      rest = g > 0.0f ? e * s : 1.0f - s;
    } else {
      s = rcp_approx(1.0f + exp2_approx(g * -1.4426950408889634f));
      rest = 1.0f - s;
    }
  }
};

template <int XT>
__device__ __forceinline__ void store16(void* p, int64_t at, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = XT == E_BF16 ? pack_bf16x2(v[2 * e], v[2 * e + 1]) : pack_f16x2(v[2 * e], v[2 * e + 1]);
  uint16_t* q = static_cast<uint16_t*>(p) + at;
  st_global_v4(q, w[0], w[1], w[2], w[3]);
  st_global_v4(q + 8, w[4], w[5], w[6], w[7]);
}

template <int FMT, int XT, bool Q>
__global__ void __launch_bounds__(kPieceThreads, 3) swiglu_backward_kernel(SwigluBackwardArgs a) {
  begin_early(true);  // its blocks move 32 KB and more
  const int items = a.N / 16;
  const int64_t p = (int64_t)blockIdx.x * kPieceThreads + threadIdx.x;
  const int64_t t = p / items;
  const int i = (int)(p - t * items);
  const bool live = t < a.rows;
  float g[16] = {}, u[16] = {};
  if (live) {
    const int64_t at = t * 2 * a.N + (int64_t)i * 16;
    float d[16] = {}, act[16];
    load16<XT>(a.h, at, g);
    load16<XT>(a.h, at + a.N, u);
    if (a.d_act) load16<XT>(a.d_act, t * a.N + (int64_t)i * 16, d);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const Sigmoid<Q && FMT == Q_BLOCKWISE> of(g[e]);
      const float silu = g[e] * of.s, ds = d[e] * of.s;
      act[e] = silu * u[e];
      const float d_g = ds * u[e] * fmaf(g[e], of.rest, 1.0f);
      u[e] = d[e] * silu;
      g[e] = d_g;
    }
    if (a.act) store16<XT>(a.act, t * a.N + (int64_t)i * 16, act);
    if (a.d_h) {
      store16<XT>(a.d_h, at, g);
      store16<XT>(a.d_h, at + a.N, u);
    }
  }
  if constexpr (Q) {
    const Quantised<FMT> og = quantise16<FMT>(g), ou = quantise16<FMT>(u);
    if (live) {
      store_codes<FMT>(og, a.q, t, i, 2 * a.N);
      store_scale<FMT>(og, a.scales, t, a.rows, i, 2 * a.N);
      store_codes<FMT>(ou, a.q, t, i + items, 2 * a.N);
      store_scale<FMT>(ou, a.scales, t, a.rows, i + items, 2 * a.N);
    }
  }
}

template <int FMT, int XT, bool Q>
cudaError_t swiglu_backward_as(const SwigluBackwardArgs& a, cudaStream_t stream) {
  const int64_t pieces = a.rows * (a.N / 16);
  const dim3 grid((unsigned)((pieces + kPieceThreads - 1) / kPieceThreads));
  return launch(swiglu_backward_kernel<FMT, XT, Q>, grid, kPieceThreads, 0, true, stream, 1, a);
}

template <int FMT>
cudaError_t swiglu_backward_format(int type, const SwigluBackwardArgs& a, cudaStream_t stream) {
  return type == E_BF16 ? swiglu_backward_as<FMT, E_BF16, true>(a, stream)
                        : swiglu_backward_as<FMT, E_FP16, true>(a, stream);
}

}  // namespace

cudaError_t launch_swiglu_backward(int format, int type, const SwigluBackwardArgs& a,
                                   cudaStream_t stream) {
  if (!a.q)
    return type == E_BF16 ? swiglu_backward_as<Q_MXFP8, E_BF16, false>(a, stream)
                          : swiglu_backward_as<Q_MXFP8, E_FP16, false>(a, stream);
  switch (format) {
    case Q_MXFP8: return swiglu_backward_format<Q_MXFP8>(type, a, stream);
    case Q_MXFP4: return swiglu_backward_format<Q_MXFP4>(type, a, stream);
    case Q_NVFP4: return swiglu_backward_format<Q_NVFP4>(type, a, stream);
    default: return swiglu_backward_format<Q_BLOCKWISE>(type, a, stream);
  }
}

}  // namespace bsfp8
