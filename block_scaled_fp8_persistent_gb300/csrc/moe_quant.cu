// Operators that write a grouped GEMM's operand: quantisation of rows (as they lie, or into
// expert order), RMS norm with the residual's addition, SwiGLU.  All are bound by HBM: each element
// is read once, its block quantised in registers (quant.cuh) and written once.
//
// What carries them is many threads with one straight piece of work each: 16 elements of a row
// per thread, one load phase, one store phase, no loop, few enough registers for 1536 to 2048
// threads per SM.  Measured against that on the same shapes: a loop over several rows per block
// with the next row's loads in flight 104 to 127 us where this takes 94 (SwiGLU, 65536 x 2048),
// tiles of 8 rows x 128 columns per warp 122.
#include <cuda_fp16.h>

#include "moe_ops.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace bsfp8 {
namespace {
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

// ---------------------------------------------------------------------------------------
// Rows of the element-wise operators: a thread takes one 16-element piece of a row.
// ---------------------------------------------------------------------------------------
constexpr int kPieceThreads = 256;
constexpr int kPieceBlocks = 6;  // per SM: at most 40 registers

// Blocks that follow a row map.  With many rows a block takes a whole row (up to 8192 elements),
// so that each copy is written in one go: 8192 rows of 7168 to 8 places in mxfp8, with their
// sort, 91 us against 97 with 224 threads.  With few rows smaller blocks reach more SMs: 16
// rows with their sort 4.1 us against 4.8.
constexpr int kMapThreads = 512;
constexpr int kMapThreadsFewRows = 128;
constexpr int64_t kMapFewRows = 512;

struct PieceGrid {
  int side;  // rows next to each other in a block, where a row alone would leave it small
  int threads;
  dim3 grid;
  PieceGrid(int64_t rows, int K, int most) {
    const int items = K / 16;
    side = items >= 64 ? 1 : 128 / items;  // (SwiGLU to 640 columns: 23.9 -> 17.5 us)
    const int parts = (items * side + most - 1) / most;  // blocks to a row
    threads = ((items * side + parts - 1) / parts + 31) / 32 * 32;
    grid = dim3((unsigned)((rows + side - 1) / side), (unsigned)parts);
  }
};

// Quantises the thread's piece (all lanes of a warp together), which load(row, item, v) fetches,
// and hands it to store(o, row, item).
template <int FMT, bool NARROW, typename Load, typename Store>
__device__ __forceinline__ void quantise_piece(int64_t rows, int items, int side, bool early,
                                               const Load& load, const Store& store) {
  begin_early(early);
  int64_t row = blockIdx.x;
  int i = blockIdx.y * blockDim.x + threadIdx.x;
  bool live = i < items;
  if constexpr (NARROW) {
    const int p = threadIdx.x / items;
    i = threadIdx.x - p * items;
    row = row * side + p;
    live = p < side && row < rows;
  }
  float v[16] = {};
  if (live) load(row, i, v);
  const Quantised<FMT> o = quantise16<FMT>(v);
  if (live) store(o, row, i);
}

// ---------------------------------------------------------------------------------------
// quantise rows; with a row map, each row goes to the rows its slots name
// ---------------------------------------------------------------------------------------
template <int FMT, int XT, bool MAP, bool NARROW>
__global__ void __launch_bounds__(MAP ? kMapThreads : kPieceThreads, MAP ? 3 : kPieceBlocks)
    quantize_kernel(QuantizeArgs a, int side, bool early) {
  quantise_piece<FMT, NARROW>(
      a.rows, a.K / 16, side, early,
      [&](int64_t t, int i, float (&v)[16]) { load16<XT>(a.x, t * a.K + (int64_t)i * 16, v); },
      [&](const Quantised<FMT>& o, int64_t t, int i) {
        if constexpr (!MAP) {
          store_codes<FMT>(o, a.q, t, i, a.K);
          store_scale<FMT>(o, a.scales, t, a.rows, i, a.K);
        } else {
          constexpr int kRows = 8;  // looked up before the stores of their copies
          for (int j0 = 0; j0 < a.top_k; j0 += kRows) {
            int row[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j)
              row[j] = j0 + j < a.top_k ? a.row_of_slot[t * a.top_k + j0 + j] : -1;
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
              if (row[j] >= a.out_rows) atomicCAS(a.err, 0, DEV_BAD_ROWS);
              if (row[j] >= 0 && row[j] < a.out_rows) {
                store_codes<FMT>(o, a.q, row[j], i, a.K);
                store_scale<FMT>(o, a.scales, row[j], a.out_rows, i, a.K);
              }
            }
          }
        }
      });
}

// 16 elements, 32-byte stores where WIDE says that p is 32-byte aligned: a lane's piece spans
// whole sectors, and 16-byte stores would write each line in several parts.
template <bool WIDE>
__device__ __forceinline__ void store16_bf16(uint16_t* p, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    st_global_v4(p, w[0], w[1], w[2], w[3]);
    st_global_v4(p + 8, w[4], w[5], w[6], w[7]);
  }
}

template <bool WIDE>
__device__ __forceinline__ void store16_fp32(float* p, const float (&v)[16]) {
  if constexpr (WIDE) {
#pragma unroll
    for (int e = 0; e < 16; e += 8)
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + e),
                   "f"(v[e]), "f"(v[e + 1]), "f"(v[e + 2]), "f"(v[e + 3]), "f"(v[e + 4]),
                   "f"(v[e + 5]), "f"(v[e + 6]), "f"(v[e + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      *reinterpret_cast<float4*>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
}

// ---------------------------------------------------------------------------------------
// RMS norm: h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight
// ---------------------------------------------------------------------------------------
//
// h stays in registers between the two passes over the row, so every input is read once.
// LANES == 0: a block per row; otherwise LANES threads of a warp per row (narrow rows).  fp32 and
// bf16 rows of 16 elements per thread are stored with 32 bytes per lane where their buffers
// allow it: with 16-byte stores each line is written in parts (16381 rows of 8192, fp32
// residual, blockwise: 234 -> 209 us, 7.1 TB/s).  bf16 residuals fit 32 registers, 2048
// threads per SM (16384 rows of 7168 with y, mxfp8: 152 us, 7.0 TB/s, against 161 with 1536);
// fp32 ones take 40 (209 against 214).
template <int FMT, bool Q, int RT, int ITEMS, bool WIDE, int LANES, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rmsnorm_kernel(NormArgs a, bool early) {
  const int64_t t = LANES ? (int64_t)blockIdx.x * (blockDim.x / (LANES ? LANES : 1)) +
                                threadIdx.x / (LANES ? LANES : 1)
                          : blockIdx.x;
  const int first = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
  const int stride = LANES ? LANES : blockDim.x;
  const int items = t < a.rows ? a.K / 16 : 0;
  begin_early(early);
  float h[ITEMS][16];
  float sum = 0.0f;
#pragma unroll
  for (int n = 0; n < ITEMS; ++n) {
    const int i = first + n * stride;
#pragma unroll
    for (int e = 0; e < 16; ++e) h[n][e] = 0.0f;
    if (i < items) {
      const int64_t at = t * a.K + (int64_t)i * 16;
      load16<E_BF16>(a.x, at, h[n]);
      if (a.residual) {
        float r[16];
        load16<RT, WIDE>(a.residual, at, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) h[n][e] += r[e];
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) sum = fmaf(h[n][e], h[n][e], sum);
      if (a.residual_out) {
        if constexpr (RT == E_FP32)
          store16_fp32<WIDE>(static_cast<float*>(a.residual_out) + at, h[n]);
        else
          store16_bf16<WIDE>(static_cast<uint16_t*>(a.residual_out) + at, h[n]);
      }
    }
  }
#pragma unroll
  for (int d = (LANES ? LANES : 32) / 2; d > 0; d /= 2)
    sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if constexpr (LANES == 0) {
    __shared__ float part[32];
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = threadIdx.x % 32 < blockDim.x / 32 ? part[threadIdx.x % 32] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  }
  const float r = rsqrtf(sum / (float)a.K + a.eps);
#pragma unroll
  for (int n = 0; n < ITEMS; ++n) {
    const int i = first + n * stride;
    if (i < items) {
      const uint4* wp =
          reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + i * 16);
      const uint4 w0 = wp[0], w1 = wp[1];
      const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float lo, hi;
        unpack_bf16x2(w[e], lo, hi);
        h[n][2 * e] *= r * lo;
        h[n][2 * e + 1] *= r * hi;
      }
      if (a.y) store16_bf16<WIDE>(static_cast<uint16_t*>(a.y) + t * a.K + (int64_t)i * 16, h[n]);
    }
    if constexpr (Q) {
      const Quantised<FMT> o = quantise16<FMT>(h[n]);
      if (i < items) {
        store_codes<FMT>(o, a.q, t, i, a.K);
        store_scale<FMT>(o, a.scales, t, a.rows, i, a.K);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// SwiGLU: g / (1 + exp(-g)) * u
// ---------------------------------------------------------------------------------------
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

// g / (1 + exp(-g)) * u for two elements.  The exponent's product with log2(e) is rounded, which
// puts |g| 2^-24 of relative error on the exponential: it matters least where |g| is large,
// beside 1 (g > 0) or in a result far below the block's largest (g < 0).  Of 100 million
// quantised elements of one sample 187 differ from the 64-bit result's, with expf 189, in plain
// fp32 227 (a few hundred that lie next to a tie: other samples turn it round); expf takes 101 us
// where this takes 92 (65536 x 2048).
__device__ __forceinline__ void swiglu2(float& g0, float& g1, float u0, float u1) {
  constexpr float kNegLog2E = -1.4426950408889634f;
  float t0, t1;
  mul2(g0, g1, kNegLog2E, kNegLog2E, t0, t1);
  const float r0 = rcp_approx(1.0f + exp2_approx(t0)), r1 = rcp_approx(1.0f + exp2_approx(t1));
  mul2(g0, g1, r0, r1, t0, t1);
  mul2(t0, t1, u0, u1, g0, g1);
}

template <int FMT, bool NARROW>
__global__ void __launch_bounds__(kPieceThreads, kPieceBlocks) swiglu_kernel(SwigluArgs a, int side,
                                                                             bool early) {
  quantise_piece<FMT, NARROW>(
      a.rows, a.N / 16, side, early,
      [&](int64_t t, int i, float (&v)[16]) {
        float u[16];
        const int64_t at = t * 2 * a.N + (int64_t)i * 16;
        load16<E_BF16>(a.h, at, v);
        load16<E_BF16>(a.h, at + a.N, u);
#pragma unroll
        for (int e = 0; e < 16; e += 2) swiglu2(v[e], v[e + 1], u[e], u[e + 1]);
      },
      [&](const Quantised<FMT>& o, int64_t t, int i) {
        store_codes<FMT>(o, a.q, t, i, a.N);
        store_scale<FMT>(o, a.scales, t, a.rows, i, a.N);
      });
}

bool aligned_32(const void* p) { return (reinterpret_cast<uintptr_t>(p) % 32) == 0; }

template <int FMT, int XT>
cudaError_t quantize_as(const QuantizeArgs& a, cudaStream_t stream) {
  const bool map = a.row_of_slot != nullptr;
  const PieceGrid g(a.rows, a.K,
                    !map                   ? kPieceThreads
                    : a.rows < kMapFewRows ? kMapThreadsFewRows
                                           : kMapThreads);
  const auto kernel = map ? (g.side > 1 ? quantize_kernel<FMT, XT, true, true>
                                        : quantize_kernel<FMT, XT, true, false>)
                          : (g.side > 1 ? quantize_kernel<FMT, XT, false, true>
                                        : quantize_kernel<FMT, XT, false, false>);
  const int each = 16 * ((XT == E_FP32 ? 4 : 2) + a.top_k);  // bytes a thread moves
  const bool early = starts_early(g.grid, (int64_t)g.threads * each);
  return launch(kernel, g.grid, g.threads, 0, early, stream, 1, a, g.side, early);
}

template <int FMT>
cudaError_t quantize_format(int x_type, const QuantizeArgs& a, cudaStream_t stream) {
  switch (x_type) {
    case E_BF16: return quantize_as<FMT, E_BF16>(a, stream);
    case E_FP16: return quantize_as<FMT, E_FP16>(a, stream);
    default: return quantize_as<FMT, E_FP32>(a, stream);
  }
}

template <int FMT, bool Q, int RT, bool WIDE>
cudaError_t norm_as(const NormArgs& a, cudaStream_t stream) {
  const int items = a.K / 16;
  const int64_t row_bytes = (int64_t)a.K * (RT == E_FP32 ? 11 : 7);  // x, residual twice, q
  const auto go = [&](void (*kernel)(NormArgs, bool), int side, int threads) {
    const unsigned blocks = (unsigned)((a.rows + side - 1) / side);
    const bool early = starts_early(blocks, side * row_bytes);
    return launch(kernel, blocks, (threads + 31) / 32 * 32, 0, early, stream, 1, a, early);
  };
  if (items <= 8) return go(rmsnorm_kernel<FMT, Q, RT, 1, WIDE, 8, 256, 8>, 32, 256);
  if (items <= 32) return go(rmsnorm_kernel<FMT, Q, RT, 1, WIDE, 32, 256, 8>, 8, 256);
  if (items <= 512)
    return go(rmsnorm_kernel<FMT, Q, RT, 1, WIDE, 0, 512, RT == E_FP32 ? 3 : 4>, 1, items);
  if (items <= 1024) return go(rmsnorm_kernel<FMT, Q, RT, 1, WIDE, 0, 1024, 2>, 1, items);
  return go(rmsnorm_kernel<FMT, Q, RT, 2, WIDE, 0, 1024, 1>, 1, (items + 1) / 2);
}

template <int FMT, bool Q>
cudaError_t norm_format(int residual_type, const NormArgs& a, cudaStream_t stream) {
  const bool w = aligned_32(a.residual) && aligned_32(a.residual_out) && aligned_32(a.y);
  if (residual_type == E_FP32)
    return w ? norm_as<FMT, Q, E_FP32, true>(a, stream) : norm_as<FMT, Q, E_FP32, false>(a, stream);
  return w ? norm_as<FMT, Q, E_BF16, true>(a, stream) : norm_as<FMT, Q, E_BF16, false>(a, stream);
}

template <int FMT>
cudaError_t swiglu_format(const SwigluArgs& a, cudaStream_t stream) {
  const PieceGrid g(a.rows, a.N, kPieceThreads);
  const bool early = starts_early(g.grid, (int64_t)g.threads * 16 * 5);
  return launch(g.side > 1 ? swiglu_kernel<FMT, true> : swiglu_kernel<FMT, false>, g.grid,
                g.threads, 0, early, stream, 1, a, g.side, early);
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
