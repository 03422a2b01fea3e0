// Launchers of the experts' products in 16 bits and of the backward pass of the experts
// (grouped16.cu, wgrad.cu, quant_columns.cu) for the C-ABI layer (capi_experts.cu), and what
// their kernels share.  Each launcher returns the launch error; sizes and alignment are checked
// by the caller.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "moe_ops.cuh"
#include "ptx.cuh"

namespace bsfp8 {

// The current device's error word and number of SMs (a bsfp8_status); capi.cu.
int device_error_word_and_sms(int** err, int* num_sms);

// Tensor map of a row-major array of `rank` dimensions, innermost first, whose box is 128 bytes
// wide and swizzled over them; what lies outside reads as zero and is not written.  Elements of
// `size` bytes: 1, 2 or 4 (fp32).  False if the driver refuses it.  capi.cu.
bool encode_swizzled(CUtensorMap* map, int size, const void* base, int rank,
                     const uint64_t* dims, uint32_t box_rows);

// Tensor map of an fp32 array [rows, cols] whose box is one row of box_cols, not swizzled.
bool encode_rows_f32(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                     uint32_t box_cols);

// C[m, n] = sum_k A[m, k] B[e, n, k], or B[e, k, n] (transposed), in bf16 or fp16.
struct Product16Args {
  const int32_t* offsets;     // [E + 1]
  const int32_t* expert_ids;  // [E], or nullptr: group e multiplies expert e
  int64_t M_total;
  int N, K;
  int E;            // groups
  int num_experts;  // experts in B
  int* err;
  const void* A;
  const void* B;
  void* C;
  bool bf16;
  bool transposed;
};
cudaError_t launch_product16(const Product16Args& a, int num_sms, cudaStream_t stream);

// The form that a product is launched in: a tile, the CTAs that compute it, how many such units share
// its K, and the K that is summed in one accumulator (0: each unit's whole part).  The sizes, type and
// direction of `a` matter only.  clusters: of 2, 4 and 8 CTAs, that a device holds at once; nullptr: the
// current one is asked.
struct Product16Plan {
  int rows, cols, ctas, split, chunk;
};
Product16Plan plan_product16(const Product16Args& a, int num_sms, const int32_t* clusters);

// dB[e, n, k] = add[e, n, k] + sum over the rows m of group e of dC[m, n] A[m, k]; e4m3 operands
// (fp8) have a scale for each block of 128 rows of a column.
enum GradType : int { GRAD_BF16 = 0, GRAD_FP16 = 1, GRAD_FP32 = 2 };
struct WgradArgs {
  const int32_t* offsets;  // [E + 1]
  int64_t M_total;
  int N, K;
  int E;
  int* err;
  const void* dC;          // [M_total, N]
  const void* A;           // [M_total, K]
  const float* dc_scales;  // fp8: [M_total / 128 + E, N]
  const float* a_scales;   // fp8: [M_total / 128 + E, K]
  const void* add;         // [E, N, K] of out_type, or nullptr
  void* dB;                // [E, N, K] of out_type
  int out_type;            // GradType
  bool fp8;
  bool bf16;               // of 16-bit operands
};
cudaError_t launch_wgrad(const WgradArgs& a, int num_sms, cudaStream_t stream);

// The form of a weight gradient: rows in a stage, pairs that share a tile's rows, and whether the
// gradients are stored by TMA.  clusters: of 8 CTAs, that a device holds at once; negative: asked.
struct WgradPlan {
  int rows, split;
  bool staged;
};
WgradPlan plan_wgrad(const WgradArgs& a, int num_sms, int64_t clusters);

// q = e4m3(x / scale) in blocks of 128 rows of a column, counted from each group's first row.
struct ColumnsArgs {
  const void* x;
  const int32_t* slot_of_row;  // [M_total], or nullptr: row r of q from row r of x
  const int32_t* offsets;      // [E + 1]
  uint8_t* q;                  // [M_total, K]
  float* scales;               // [M_total / 128 + E, K]
  int64_t M_total, x_rows;
  int top_k, K, E;
  int* err;
};
cudaError_t launch_quantize_columns(int x_type, const ColumnsArgs& a, cudaStream_t stream);

// Launches a persistent kernel in clusters of `cluster` blocks, one block to an SM.  It starts while
// the one before it on the stream is still running (moe_ops.cuh): barriers, tensor memory and
// tensor maps are ready by the time its inputs are.  It lets the next one do so once it has its
// tensor memory, so that no kernel that waits for it can hold what it needs.
template <typename... Params, typename... Args>
cudaError_t launch_persistent(void (*kernel)(Params...), int64_t units, int cluster, int threads,
                              size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = cluster;
  attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cluster));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A kernel's limit of dynamic shared memory, set once per device (several host threads may call).
template <auto kernel>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<bool> set[64];
  int dev = 0;
  const cudaError_t got = cudaGetDevice(&dev);
  if (got != cudaSuccess) return got;
  if (dev < 64 && set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) set[dev].store(true, std::memory_order_release);
  return e;
}

// How many clusters of `cluster` blocks of a kernel the device holds at once (SMs of a cluster are
// of one GPC, so some stay over: of 152 SMs 36 clusters of 4, 15 of 8), asked once per device.
template <auto kernel>
int64_t clusters_at_once(int cluster, int threads, size_t smem) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64) {
    const int n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n - 1;
  }
  if (allow_smem<kernel>(smem) != cudaSuccess) return 0;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

// ---------------------------------------------------------------------------------------
// device side
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ void give_up(int* err, volatile int* abort) {
  atomicCAS(err, 0, (int)DEV_TIMEOUT);
  *abort = 1;
}

}  // namespace bsfp8
