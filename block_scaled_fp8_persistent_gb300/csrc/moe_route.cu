// Tokens sorted by expert, and the way back: the stable counting sort that gives every slot
// (token t's j-th choice, slot t * top_k + j) its row in the grouped GEMM's operand, the
// weighted sum of a token's rows, and that sum's gradient.
#include "common.cuh"
#include "moe_ops.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace bsfp8 {
namespace {

// ---------------------------------------------------------------------------------------
// counting sort
//
// The slots are cut into chunks of one block each and a block's part into one contiguous
// segment per warp.  A slot's row is
//   (slots of smaller keys) + (slots of its key in earlier chunks) + (in earlier warps)
//   + (earlier in its warp),
// the key being the expert, or `experts` for dropped slots.  Counts only, no atomics whose
// order could show: equal keys keep their order.
// ---------------------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortMaxChunks = 128;
constexpr int kSortChunk = 1024;       // smallest chunk: one 32-slot step per warp
constexpr int64_t kSortSingle = 4096;  // up to here one block sorts alone
constexpr int kSortSmemWords = 40 * 1024;

int64_t sort_chunk(int64_t slots) {
  const int64_t c = (slots + kSortMaxChunks - 1) / kSortMaxChunks;
  return (c + kSortChunk - 1) / kSortChunk * kSortChunk;
}

int sort_warps(int64_t chunk, int experts) {
  int w = kSortThreads / 32;
  while (w > 1 && w * (experts + 1) > kSortSmemWords) w /= 2;
  while (w > 1 && (w / 2) * 32 >= chunk) w /= 2;
  return w;
}

__device__ __forceinline__ int key_of(int id, int experts) {
  return (unsigned)id < (unsigned)experts ? id : experts;
}

// Counts per key of one chunk: counts[chunk * keys + key].
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a, int64_t chunk) {
  extern __shared__ int hist[];
  const int keys = a.experts + 1;
  for (int e = threadIdx.x; e < keys; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * chunk;
  const int64_t end = begin + chunk < a.slots ? begin + chunk : a.slots;
  for (int64_t s = begin + threadIdx.x; s < end; s += blockDim.x)
    atomicAdd(&hist[key_of(__ldg(a.ids + s), a.experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += blockDim.x)
    a.workspace[(int64_t)blockIdx.x * keys + e] = hist[e];
}

// Exclusive prefix sum of one value per thread over the block, and the block's total.
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  const int warps = blockDim.x / 32;
  int w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
  __syncthreads();
  return before + inc - v;
}

// Rows of one chunk's slots.  With one block the counts come from its own histograms,
// otherwise from the counts of every chunk.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a, int64_t chunk,
                                                                  int warps) {
  extern __shared__ int hist[];  // [warps][keys]
  __shared__ int warp_sums[32];
  const int keys = a.experts + 1;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t begin = blockIdx.x * chunk;
  const int64_t end = begin + chunk < a.slots ? begin + chunk : a.slots;
  const int64_t seg = ((end - begin + warps - 1) / warps + 31) / 32 * 32;
  const int64_t lo = begin + warp * seg;
  const int64_t hi = warp < warps ? (lo + seg < end ? lo + seg : end) : lo;

  for (int e = threadIdx.x; e < warps * keys; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  for (int64_t s = lo + lane; s < hi; s += 32)
    atomicAdd(&hist[warp * keys + key_of(__ldg(a.ids + s), a.experts)], 1);
  __syncthreads();

  int carry = 0;
  for (int e0 = 0; e0 < keys; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int mine = 0, before = 0, all = 0;
    if (e < keys) {
      for (int w = 0; w < warps; ++w) {
        const int c = hist[w * keys + e];
        hist[w * keys + e] = mine;
        mine += c;
      }
      all = mine;
      if (gridDim.x > 1) {
        all = 0;
#pragma unroll 16
        for (int b = 0; b < (int)gridDim.x; ++b) {
          const int c = __ldg(a.workspace + (int64_t)b * keys + e);
          all += c;
          if (b < (int)blockIdx.x) before += c;
        }
      }
    }
    int total;
    const int first = carry + block_exclusive(all, warp_sums, total);
    carry += total;
    if (e < keys) {
      for (int w = 0; w < warps; ++w) hist[w * keys + e] += first + before;
      if (blockIdx.x == 0) a.offsets[e] = first;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[keys] = (int)a.slots;
  __syncthreads();

  for (int64_t s0 = lo; s0 < hi; s0 += 32) {
    const int64_t s = s0 + lane;
    const bool live = s < hi;
    const unsigned active = __ballot_sync(0xffffffffu, live);
    if (live) {
      const int key = key_of(__ldg(a.ids + s), a.experts);
      const unsigned peers = __match_any_sync(active, key);
      const int rank = __popc(peers & ((1u << lane) - 1));
      int* h = &hist[warp * keys + key];
      const int row = *h + rank;
      __syncwarp(active);
      if (rank == 0) *h = row + __popc(peers);
      __syncwarp(active);
      a.row_of_slot[s] = key < a.experts ? row : -1;
      if (a.slot_of_row) a.slot_of_row[row] = key < a.experts ? (int)s : -1;
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------------------
// weighted sum of a token's rows, and its gradient
// ---------------------------------------------------------------------------------------
constexpr int kSlots = 8;  // rows in flight per thread

__device__ __forceinline__ int checked_row(const int32_t* row_of_slot, int64_t slot,
                                           int64_t in_rows, int* err) {
  const int row = __ldg(row_of_slot + slot);
  if (row >= in_rows) {
    atomicCAS(err, 0, DEV_BAD_ROWS);
    return -1;
  }
  return row;
}

__device__ __forceinline__ void unpack8(const uint32_t (&w)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_bf16x2(w[i], v[2 * i], v[2 * i + 1]);
}

__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a) {
  const int64_t t = blockIdx.x;
  const int col = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
  if (col >= a.N) return;
  float acc[8] = {};
  if (a.residual) {
    uint32_t w[4];
    load_stream<4, false>(static_cast<const uint16_t*>(a.residual) + t * a.N + col, w);
    unpack8(w, acc);
  }
  for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
    uint32_t w[kSlots][4];
    int row[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      row[j] = j0 + j < a.top_k
                   ? checked_row(a.row_of_slot, t * a.top_k + j0 + j, a.in_rows, a.err)
                   : -1;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (row[j] >= 0)
        load_stream<4, false>(static_cast<const uint16_t*>(a.C) + (int64_t)row[j] * a.N + col, w[j]);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (row[j] >= 0) {
        const float g = a.weights ? __ldg(a.weights + t * a.top_k + j0 + j) : 1.0f;
        float v[8];
        unpack8(w[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(g, v[e], acc[e]);
      }
    }
  }
  st_global_v4(static_cast<uint16_t*>(a.out) + t * a.N + col, pack_bf16x2(acc[0], acc[1]),
               pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
               pack_bf16x2(acc[6], acc[7]));
}

__global__ void __launch_bounds__(256) combine_backward_kernel(CombineBackwardArgs a) {
  __shared__ float part[8][kSlots];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int j0 = 0; j0 < a.top_k; j0 += kSlots) {
    int row[kSlots];
    float g[kSlots], dot[kSlots] = {};
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const bool there = j0 + j < a.top_k;
      row[j] = there ? checked_row(a.row_of_slot, t * a.top_k + j0 + j, a.in_rows, a.err) : -1;
      g[j] = there ? __ldg(a.weights + t * a.top_k + j0 + j) : 0.0f;
    }
    for (int col = threadIdx.x * 8; col < a.N; col += blockDim.x * 8) {
      uint32_t wd[4], w[kSlots][4];
      float d[8];
      load_stream<4, false>(static_cast<const uint16_t*>(a.d_out) + t * a.N + col, wd);
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (row[j] >= 0)
          load_stream<4, false>(static_cast<const uint16_t*>(a.C) + (int64_t)row[j] * a.N + col, w[j]);
      unpack8(wd, d);
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        if (row[j] < 0) continue;
        float v[8];
        unpack8(w[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot[j] = fmaf(d[e], v[e], dot[j]);
        st_global_v4(static_cast<uint16_t*>(a.dC) + (int64_t)row[j] * a.N + col,
                     pack_bf16x2(g[j] * d[0], g[j] * d[1]), pack_bf16x2(g[j] * d[2], g[j] * d[3]),
                     pack_bf16x2(g[j] * d[4], g[j] * d[5]), pack_bf16x2(g[j] * d[6], g[j] * d[7]));
      }
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o /= 2) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < a.top_k) {
      float s = 0.0f;
      for (int w = 0; w < (int)blockDim.x / 32; ++w) s += part[w][threadIdx.x];
      a.d_weights[t * a.top_k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

}  // namespace

int64_t moe_sort_workspace_bytes(int64_t slots, int experts) {
  if (slots <= kSortSingle) return 0;
  const int64_t chunk = sort_chunk(slots);
  return (slots + chunk - 1) / chunk * (experts + 1) * (int64_t)sizeof(int32_t);
}

cudaError_t launch_moe_sort(const SortArgs& a, cudaStream_t stream) {
  const int keys = a.experts + 1;
  const bool single = a.slots <= kSortSingle;
  const int64_t chunk = single ? a.slots : sort_chunk(a.slots);
  const int chunks = single ? 1 : (int)((a.slots + chunk - 1) / chunk);
  const int warps = sort_warps(chunk, a.experts);
  // one thread per key in the scan, as far as a block goes
  int threads = (keys + 31) / 32 * 32;
  threads = threads < warps * 32 ? warps * 32 : threads;
  threads = threads < kSortThreads ? threads : kSortThreads;
  const size_t smem = (size_t)warps * keys * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmemWords * 4);
    if (e != cudaSuccess) return e;
  }
  if (!single) {
    sort_count_kernel<<<chunks, kSortThreads, keys * sizeof(int), stream>>>(a, chunk);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  sort_place_kernel<<<chunks, threads, smem, stream>>>(a, chunk, warps);
  return cudaGetLastError();
}

cudaError_t launch_moe_combine(const CombineArgs& a, cudaStream_t stream) {
  const int vecs = a.N / 8;
  const int threads = vecs >= 256 ? 256 : (vecs + 31) / 32 * 32;
  const dim3 grid((unsigned)a.rows, (unsigned)((vecs + threads - 1) / threads));
  combine_kernel<<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_moe_combine_backward(const CombineBackwardArgs& a, cudaStream_t stream) {
  const int vecs = a.N / 8;
  const int threads = vecs >= 256 ? 256 : (vecs + 31) / 32 * 32;
  combine_backward_kernel<<<(unsigned)a.rows, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace bsfp8
