// C-ABI entry points of the experts' products in 16 bits and of the backward pass of the experts:
// argument checks on the host, then one launch.  The contract lives in include/bsfp8.h.
#include "bsfp8.h"
#include "expert_ops.cuh"
#include "moe_ops.cuh"

using namespace bsfp8;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool rows_ok(int64_t rows) { return rows >= 0 && rows <= INT32_MAX; }
// of groups: a row past a group's last tile is still an int
bool grouped_rows_ok(int64_t rows) { return rows >= 0 && rows <= INT32_MAX - 1024; }

constexpr int kMaxWidth = 1 << 24;
constexpr int kMaxGroups = 1 << 20;
bool groups_ok(int groups) { return groups >= 1 && groups <= kMaxGroups; }

// sides of a matrix in multiples of `step`; its bytes stay within a tensor map's strides
bool matrix_ok(int N, int K, int step) {
  return N >= step && N % step == 0 && N <= kMaxWidth && K >= step && K % step == 0 &&
         K <= kMaxWidth && (int64_t)N * K < ((int64_t)1 << 38);
}

bsfp8_status launched(cudaError_t e) { return e == cudaSuccess ? BSFP8_OK : BSFP8_ERR_CUDA; }

bool half_type(int type) { return type == BSMX_BF16 || type == BSMX_FP16; }

bsfp8_status wgrad(const WgradArgs& a, int step, cudaStream_t stream) {
  if (!a.offsets || !a.dB ||
      (a.M_total > 0 && (!a.dC || !a.A || (a.fp8 && (!a.dc_scales || !a.a_scales)))))
    return BSFP8_ERR_NULL;
  if (!grouped_rows_ok(a.M_total) || !matrix_ok(a.N, a.K, step) || !groups_ok(a.E)) return BSFP8_ERR_SHAPE;
  if (!aligned(a.dC, 16) || !aligned(a.A, 16) || !aligned(a.dB, 16) || !aligned(a.add, 16) ||
      !aligned(a.dc_scales, 16) || !aligned(a.a_scales, 16) || !aligned(a.offsets, 4))
    return BSFP8_ERR_ALIGN;
  WgradArgs go = a;
  int sms = 0;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word_and_sms(&go.err, &sms));
  if (st != BSFP8_OK) return st;
  return launched(launch_wgrad(go, sms, stream));
}

}  // namespace

extern "C" bsfp8_status bs16_grouped_gemm(int type, int transposed, const void* A, const void* B,
                                          const int32_t* group_offsets, const int32_t* expert_ids,
                                          void* C, int64_t M_total, int N, int K, int num_groups,
                                          int num_experts, cudaStream_t stream) {
  if (!half_type(type)) return BSFP8_ERR_FORMAT;
  if (!group_offsets || !B || (M_total > 0 && (!A || !C))) return BSFP8_ERR_NULL;
  if (!grouped_rows_ok(M_total) || !matrix_ok(N, K, 8) || !groups_ok(num_groups) ||
      !groups_ok(num_experts) || (!expert_ids && num_groups > num_experts))
    return BSFP8_ERR_SHAPE;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(group_offsets, 4) ||
      !aligned(expert_ids, 4))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  int sms = 0;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word_and_sms(&err, &sms));
  if (st != BSFP8_OK) return st;
  if (M_total == 0) return BSFP8_OK;
  return launched(launch_product16(
      Product16Args{group_offsets, expert_ids, M_total, N, K, num_groups, num_experts, err,
                    A, B, C, type == BSMX_BF16, transposed != 0},
      sms, stream));
}

extern "C" bsfp8_status bs16_grouped_gemm_plan(int type, int transposed, int64_t M_total, int N,
                                               int K, int num_groups, int num_sms,
                                               const int32_t* clusters, int32_t* out) {
  if (!out) return BSFP8_ERR_NULL;
  if (!half_type(type)) return BSFP8_ERR_FORMAT;
  if (M_total < 1 || !grouped_rows_ok(M_total) || !matrix_ok(N, K, 8) || !groups_ok(num_groups) ||
      num_sms < 2)
    return BSFP8_ERR_SHAPE;
  const Product16Plan p = plan_product16(
      Product16Args{nullptr, nullptr, M_total, N, K, num_groups, num_groups, nullptr, nullptr,
                    nullptr, nullptr, type == BSMX_BF16, transposed != 0},
      num_sms, clusters);
  const int32_t form[5] = {p.rows, p.cols, p.ctas, p.split, p.chunk};
  for (int i = 0; i < 5; ++i) out[i] = form[i];
  return BSFP8_OK;
}

extern "C" bsfp8_status bs16_grouped_wgrad(int type, int out_type, const void* dC, const void* A,
                                           const int32_t* group_offsets, const void* add, void* dB,
                                           int64_t M_total, int N, int K, int num_experts,
                                           cudaStream_t stream) {
  if (!half_type(type) || (out_type != type && out_type != BSMX_FP32)) return BSFP8_ERR_FORMAT;
  return wgrad(WgradArgs{group_offsets, M_total, N, K, num_experts, nullptr, dC, A, nullptr,
                         nullptr, add, dB, out_type, false, type == BSMX_BF16},
               8, stream);
}

extern "C" bsfp8_status bsfp8_grouped_wgrad(int out_type, const void* dC, const void* A,
                                            const float* dc_scales, const float* a_scales,
                                            const int32_t* group_offsets, const void* add,
                                            void* dB, int64_t M_total, int N, int K,
                                            int num_experts, cudaStream_t stream) {
  if (out_type < BSMX_BF16 || out_type > BSMX_FP32) return BSFP8_ERR_FORMAT;
  return wgrad(WgradArgs{group_offsets, M_total, N, K, num_experts, nullptr, dC, A, dc_scales,
                         a_scales, add, dB, out_type, true, false},
               128, stream);
}

extern "C" bsfp8_status bsfp8_grouped_wgrad_plan(int fp8, int out_type, int added,
                                                 int64_t M_total, int N, int K, int num_experts,
                                                 int num_sms, int clusters_of_8, int32_t* out) {
  if (!out) return BSFP8_ERR_NULL;
  if (out_type < BSMX_BF16 || out_type > BSMX_FP32) return BSFP8_ERR_FORMAT;
  if (!grouped_rows_ok(M_total) || !matrix_ok(N, K, fp8 ? 128 : 8) || !groups_ok(num_experts) ||
      num_sms < 2)
    return BSFP8_ERR_SHAPE;
  WgradArgs a{};
  a.M_total = M_total;
  a.N = N;
  a.K = K;
  a.E = num_experts;
  a.out_type = out_type;
  a.fp8 = fp8 != 0;
  a.add = added ? &a : nullptr;  // (only whether there is one counts)
  const WgradPlan p = plan_wgrad(a, num_sms, clusters_of_8);
  const int32_t form[3] = {p.rows, p.split, p.staged};
  for (int i = 0; i < 3; ++i) out[i] = form[i];
  return BSFP8_OK;
}

extern "C" bsfp8_status bsfp8_quantize_columns(int x_type, const void* x,
                                               const int32_t* slot_of_row, int top_k,
                                               const int32_t* group_offsets, void* q,
                                               float* scales, int64_t M_total, int64_t x_rows,
                                               int K, int num_groups, cudaStream_t stream) {
  if (x_type < BSMX_BF16 || x_type > BSMX_FP32) return BSFP8_ERR_FORMAT;
  if (!group_offsets || (M_total > 0 && (!q || !scales || (x_rows > 0 && !x))))
    return BSFP8_ERR_NULL;
  if (!grouped_rows_ok(M_total) || !rows_ok(x_rows) || K < 128 || K % 128 != 0 || K > (1 << 22) ||
      !groups_ok(num_groups) || top_k < 1 || top_k > 64 ||
      (M_total > 0 && !slot_of_row && (top_k != 1 || x_rows != M_total)))
    return BSFP8_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 16) || !aligned(slot_of_row, 4) ||
      !aligned(group_offsets, 4))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  if (M_total == 0) return BSFP8_OK;
  return launched(launch_quantize_columns(
      x_type,
      ColumnsArgs{x, slot_of_row, group_offsets, static_cast<uint8_t*>(q), scales, M_total, x_rows,
                  top_k, K, num_groups, err},
      stream));
}

extern "C" bsfp8_status bsmx_swiglu_backward(int type, int format, const void* h,
                                             const void* d_act, void* d_h, void* act, void* q,
                                             void* scales, int64_t rows, int N,
                                             cudaStream_t stream) {
  if (!half_type(type) || format < BSMX_MXFP8 || format > BSMX_BLOCKWISE) return BSFP8_ERR_FORMAT;
  if (rows > 0 && (!h || (!d_h && !act && !q) || ((d_h || q) && !d_act) || (q && !scales)))
    return BSFP8_ERR_NULL;
  if (!rows_ok(rows) || N < 128 || N % 128 != 0 || N > kMaxWidth / 2 ||
      rows * (N / 128) > ((int64_t)1 << 35))
    return BSFP8_ERR_SHAPE;
  if (!aligned(h, 16) || !aligned(d_act, 16) || !aligned(d_h, 16) || !aligned(act, 16) ||
      !aligned(q, 16) || (format == BSMX_BLOCKWISE && !aligned(scales, 4)))
    return BSFP8_ERR_ALIGN;
  int* err = nullptr;
  const bsfp8_status st = static_cast<bsfp8_status>(device_error_word(&err));
  if (st != BSFP8_OK) return st;
  if (rows == 0) return BSFP8_OK;
  return launched(launch_swiglu_backward(
      format, type,
      SwigluBackwardArgs{h, d_act, d_h, act, static_cast<uint8_t*>(q), scales, rows, N}, stream));
}
