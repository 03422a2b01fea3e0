// Launchers of the operators around the grouped GEMM (moe_quant.cu, moe_route.cu) for the
// C-ABI layer (capi_moe.cu).  Each returns the launch error; sizes and alignment are checked
// by the caller.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace bsfp8 {

// Programmatic launches.  A kernel of these operators starts while the one before it on the
// stream is still running: it lets the next one do so, and touches memory only once the kernel
// before has completed and its writes are visible (at once where that one was not overlapped).
// No load of these kernels takes the read-only path: what they read may be written by a kernel
// that runs after they were launched.  Back to back on a stream that saves 2 to 3 us of every
// launch of 15 to 200 us, and 0.3 us of 2 to 3 at decode size.  The two instructions also cost
// each block some time, so grids of many blocks with little to do go without (`early` false):
// 8192 x 2 rows of 512 columns summed 6.9 us without, 8.9 with; 16384 rows of 640 normed 16.2
// and 17.9.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void begin_early(bool early) {
  if (early) {
    launch_dependents();
    wait_for_previous();
  }
}

constexpr uint64_t kEarlyBlocks = 1024;  // up to here a grid starts early,
constexpr int64_t kEarlyBytes = 8192;    // or where its blocks move this much each
inline bool starts_early(dim3 grid, int64_t block_bytes) {
  return (uint64_t)grid.x * grid.y <= kEarlyBlocks || block_bytes >= kEarlyBytes;
}

// cluster: blocks of one, all of a grid's where it is above 1
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, bool early,
                   cudaStream_t stream, int cluster, A... args) {
  cudaLaunchAttribute attrs[2] = {};
  unsigned n = 0;
  if (early) {
    attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attrs[n].id = cudaLaunchAttributeClusterDimension;
    attrs[n].val.clusterDim.x = cluster;
    attrs[n].val.clusterDim.y = attrs[n].val.clusterDim.z = 1;
    ++n;
  }
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = block;
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = attrs;
  config.numAttrs = n;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

// Device error code beside those of common.cuh: a row map's entry names a row that is not there.
constexpr int DEV_BAD_ROWS = 11;

// The current device's error word (a bsfp8_status: BSFP8_OK, or why there is none); capi.cu.
int device_error_word(int** err);

enum ElementType : int { E_BF16 = 0, E_FP16 = 1, E_FP32 = 2 };

struct QuantizeArgs {
  const void* x;               // [rows, K]
  const int32_t* row_of_slot;  // [rows * top_k], or nullptr: row t of q from row t of x
  uint8_t* q;
  void* scales;
  int64_t rows, out_rows;
  int top_k, K;
  int* err;
};
cudaError_t launch_quantize(int format, int x_type, const QuantizeArgs& a, cudaStream_t stream);

struct NormArgs {
  const void* x;         // bf16 [rows, K]
  const void* residual;  // bf16 or fp32 [rows, K], or nullptr
  const void* weight;    // bf16 [K]
  void* residual_out;    // as residual, or nullptr
  void* y;               // bf16 [rows, K], or nullptr
  uint8_t* q;            // or nullptr
  void* scales;
  int64_t rows;
  int K;
  float eps;
};
constexpr int kNormMaxK = 32768;
cudaError_t launch_rmsnorm_quant(int format, int residual_type, const NormArgs& a,
                                 cudaStream_t stream);

struct SwigluArgs {
  const void* h;  // bf16 [rows, 2N], gate then up
  uint8_t* q;
  void* scales;
  int64_t rows;
  int N;
};
cudaError_t launch_swiglu_quant(int format, const SwigluArgs& a, cudaStream_t stream);

struct SwigluBackwardArgs {
  const void* h;      // [rows, 2N], gate then up
  const void* d_act;  // [rows, N], or nullptr: act only
  void* d_h;          // [rows, 2N], or nullptr
  void* act;          // [rows, N], or nullptr
  uint8_t* q;         // of d_h, or nullptr
  void* scales;
  int64_t rows;
  int N;
};
cudaError_t launch_swiglu_backward(int format, int type, const SwigluBackwardArgs& a,
                                   cudaStream_t stream);

struct SortArgs {
  const int32_t* ids;    // [slots]
  int32_t* offsets;      // [experts + 2]
  int32_t* row_of_slot;  // [slots]
  int32_t* slot_of_row;  // [slots], or nullptr
  int32_t* workspace;
  int64_t slots;
  int experts;
};
constexpr int kSortMaxExperts = 4096;
int64_t moe_sort_workspace_bytes(int64_t slots, int experts);
cudaError_t launch_moe_sort(const SortArgs& a, cudaStream_t stream);

struct CombineArgs {
  const void* C;               // bf16 [in_rows, N]
  const int32_t* row_of_slot;  // [rows * top_k]
  const float* weights;        // [rows * top_k], or nullptr: 1
  const void* residual;        // bf16 [rows, N], or nullptr
  void* out;                   // bf16 [rows, N]
  int64_t rows, in_rows;
  int top_k, N;
  int* err;
};
cudaError_t launch_moe_combine(const CombineArgs& a, cudaStream_t stream);

struct CombineBackwardArgs {
  const void* d_out;           // bf16 [rows, N]
  const void* C;               // bf16 [in_rows, N]
  const int32_t* row_of_slot;  // [rows * top_k]
  const float* weights;        // [rows * top_k]
  void* dC;                    // bf16 [in_rows, N]
  float* d_weights;            // [rows * top_k]
  int64_t rows, in_rows;
  int top_k, N;
  int* err;
};
cudaError_t launch_moe_combine_backward(const CombineBackwardArgs& a, cudaStream_t stream);

}  // namespace bsfp8
