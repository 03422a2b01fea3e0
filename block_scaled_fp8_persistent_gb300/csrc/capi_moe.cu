// C-ABI entry points of the operators around the grouped GEMM: argument checks on the host,
// then one launch (two for a sort of many slots).  The contract lives in include/bsfp8.h.
#include <cmath>

#include "bsfp8.h"
#include "moe_ops.cuh"

using namespace bsfp8;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool format_ok(int format) { return format >= BSMX_MXFP8 && format <= BSMX_BLOCKWISE; }

bool rows_ok(int64_t rows) { return rows >= 0 && rows <= INT32_MAX; }

// widths up to 2^24, so that a row's blocks fit the grid
constexpr int kMaxWidth = 1 << 24;
bool width_ok(int K) { return K >= 128 && K % 128 == 0 && K <= kMaxWidth; }

constexpr int kMaxTopK = 64;

bool columns_ok(int N) { return N >= 8 && N % 8 == 0 && N <= kMaxWidth; }

bool slots_ok(int64_t rows, int top_k) {
  return rows_ok(rows) && top_k >= 1 && top_k <= kMaxTopK && rows * top_k <= INT32_MAX;
}

// codes and scales of an operand in `format`
bool operand_aligned(int format, const void* q, const void* scales) {
  return aligned(q, 16) && aligned(scales, format == BSMX_BLOCKWISE ? 4 : 1);
}

bsfp8_status launched(cudaError_t e) { return e == cudaSuccess ? BSFP8_OK : BSFP8_ERR_CUDA; }

}  // namespace

extern "C" bsfp8_status bsmx_quantize(int format, int x_type, const void* x,
                                      const int32_t* row_of_slot, int top_k, void* q,
                                      void* scales, int64_t rows, int64_t out_rows, int K,
                                      cudaStream_t stream) {
  if (!format_ok(format) || x_type < BSMX_BF16 || x_type > BSMX_FP32) return BSFP8_ERR_FORMAT;
  if (rows > 0 && (!x || !q || !scales)) return BSFP8_ERR_NULL;
  if (!width_ok(K) || !slots_ok(rows, top_k) || !rows_ok(out_rows) ||
      (rows > 0 && !row_of_slot && (top_k != 1 || out_rows != rows)))
    return BSFP8_ERR_SHAPE;
  if (!aligned(x, 16) || !operand_aligned(format, q, scales) || !aligned(row_of_slot, 4))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  if (rows == 0) return BSFP8_OK;
  return launched(launch_quantize(
      format, x_type,
      QuantizeArgs{x, row_of_slot, static_cast<uint8_t*>(q), scales, rows, out_rows, top_k, K, err},
      stream));
}

extern "C" bsfp8_status bsmx_rmsnorm_quant(int format, int residual_type, const void* x,
                                           const void* residual, const void* weight, float eps,
                                           void* residual_out, void* y, void* q, void* scales,
                                           int64_t rows, int K, cudaStream_t stream) {
  if (!format_ok(format) || (residual_type != BSMX_BF16 && residual_type != BSMX_FP32))
    return BSFP8_ERR_FORMAT;
  if (!weight || (rows > 0 && (!x || (!y && !q && !residual_out) || (q && !scales))))
    return BSFP8_ERR_NULL;
  if (!width_ok(K) || K > kNormMaxK || !rows_ok(rows) || !(eps > 0.0f) || !std::isfinite(eps))
    return BSFP8_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
      !aligned(residual_out, 16) || !aligned(y, 16) || !operand_aligned(format, q, scales))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  if (rows == 0) return BSFP8_OK;
  return launched(launch_rmsnorm_quant(format, residual_type,
                                       NormArgs{x, residual, weight, residual_out, y,
                                                static_cast<uint8_t*>(q), scales, rows, K, eps},
                                       stream));
}

extern "C" bsfp8_status bsmx_swiglu_quant(int format, const void* h, void* q, void* scales,
                                          int64_t rows, int N, cudaStream_t stream) {
  if (!format_ok(format)) return BSFP8_ERR_FORMAT;
  if (rows > 0 && (!h || !q || !scales)) return BSFP8_ERR_NULL;
  if (!width_ok(N) || !rows_ok(rows)) return BSFP8_ERR_SHAPE;
  if (!aligned(h, 16) || !operand_aligned(format, q, scales)) return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  if (rows == 0) return BSFP8_OK;
  return launched(launch_swiglu_quant(
      format, SwigluArgs{h, static_cast<uint8_t*>(q), scales, rows, N}, stream));
}

extern "C" bsfp8_status bsmx_moe_sort_workspace(int64_t rows, int top_k, int num_experts,
                                                int64_t* bytes) {
  if (!bytes) return BSFP8_ERR_NULL;
  if (!slots_ok(rows, top_k) || num_experts < 1 || num_experts > kSortMaxExperts)
    return BSFP8_ERR_SHAPE;
  *bytes = moe_sort_workspace_bytes(rows * top_k, num_experts);
  return BSFP8_OK;
}

extern "C" bsfp8_status bsmx_moe_sort(const int32_t* topk_ids, int32_t* offsets,
                                      int32_t* row_of_slot, int32_t* slot_of_row,
                                      void* workspace, int64_t workspace_bytes, int64_t rows,
                                      int top_k, int num_experts, cudaStream_t stream) {
  if (!offsets || (rows > 0 && (!topk_ids || !row_of_slot))) return BSFP8_ERR_NULL;
  int64_t need = 0;
  const bsfp8_status shape = bsmx_moe_sort_workspace(rows, top_k, num_experts, &need);
  if (shape != BSFP8_OK) return shape;
  if (need > 0 && !workspace) return BSFP8_ERR_NULL;
  if (workspace_bytes < need) return BSFP8_ERR_SHAPE;
  if (!aligned(topk_ids, 4) || !aligned(offsets, 4) || !aligned(row_of_slot, 4) ||
      !aligned(slot_of_row, 4) || !aligned(workspace, 4))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  return launched(launch_moe_sort(SortArgs{topk_ids, offsets, row_of_slot, slot_of_row,
                                           static_cast<int32_t*>(workspace), rows * top_k,
                                           num_experts},
                                  stream));
}

extern "C" bsfp8_status bsmx_moe_combine(const void* C, const int32_t* row_of_slot,
                                         const float* weights, const void* residual, void* out,
                                         int64_t rows, int64_t in_rows, int top_k, int N,
                                         cudaStream_t stream) {
  if (rows > 0 && (!row_of_slot || !out || (in_rows > 0 && !C))) return BSFP8_ERR_NULL;
  if (!slots_ok(rows, top_k) || !rows_ok(in_rows) || !columns_ok(N)) return BSFP8_ERR_SHAPE;
  if (!aligned(C, 16) || !aligned(residual, 16) || !aligned(out, 16) ||
      !aligned(row_of_slot, 4) || !aligned(weights, 4))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  if (rows == 0) return BSFP8_OK;
  return launched(launch_moe_combine(
      CombineArgs{C, row_of_slot, weights, residual, out, rows, in_rows, top_k, N, err}, stream));
}

extern "C" bsfp8_status bsmx_moe_combine_backward(const void* d_out, const void* C,
                                                  const int32_t* row_of_slot,
                                                  const float* weights, void* dC,
                                                  float* d_weights, int64_t rows,
                                                  int64_t in_rows, int top_k, int N,
                                                  cudaStream_t stream) {
  if (rows > 0 && (!d_out || !row_of_slot || !weights || !d_weights || (in_rows > 0 && (!C || !dC))))
    return BSFP8_ERR_NULL;
  if (!slots_ok(rows, top_k) || !rows_ok(in_rows) || !columns_ok(N)) return BSFP8_ERR_SHAPE;
  if (!aligned(d_out, 16) || !aligned(C, 16) || !aligned(dC, 16) || !aligned(row_of_slot, 4) ||
      !aligned(weights, 4) || !aligned(d_weights, 4))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  if (rows == 0) return BSFP8_OK;
  return launched(launch_moe_combine_backward(
      CombineBackwardArgs{d_out, C, row_of_slot, weights, dC, d_weights, rows, in_rows, top_k, N, err},
      stream));
}
