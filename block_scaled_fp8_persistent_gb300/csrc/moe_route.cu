// Tokens sorted by expert, and the way back: the stable counting sort that gives every slot
// (token t's j-th choice, slot t * top_k + j) its row in the grouped GEMM's operand, the
// weighted sum of a token's rows, and that sum's gradient.
#include <atomic>

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
// order could show: equal keys keep their order.  Bound by launches and round trips to L2, not
// by bytes (12 per slot).  64 / 256 experts: one block up to kSortSingle slots (128 slots 1.9 us,
// 512 slots 2.4; 1024 would take 3.3 / 3.7); a cluster of eight, whose blocks read each other's
// counts from shared memory, up to kSortCluster (1024 slots 2.8 / 3.2 us, 4096 slots 3.6 / 3.9,
// 16384 slots 5.4 / 6.2; 65536 would take 11.1 / 12.4); above that many blocks and two launches,
// the second started before the first ends (8192 would take 5.7 / 7.1, 16384 slots 5.9 / 7.3;
// 65536 slots 5.9 / 7.7, 524288 slots 9.1 / 11.5; back to back in a graph).
// ---------------------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortMaxChunks = 128;
constexpr int kSortChunk = 1024;         // smallest chunk: one 32-slot step per warp
constexpr int64_t kSortSingle = 512;     // up to here one block sorts alone
constexpr int64_t kSortCluster = 16384;  // up to here one cluster
constexpr int kSortClusterBlocks = 8;
constexpr int kSortSmemWords = 40 * 1024;

int64_t sort_chunk(int64_t slots) {
  const int64_t c = (slots + kSortMaxChunks - 1) / kSortMaxChunks;
  return (c + kSortChunk - 1) / kSortChunk * kSortChunk;
}

// Words from one warp's counts to the next: odd, so that the 32 warps' counts of one key lie
// in 32 banks.
__host__ __device__ __forceinline__ int sort_pitch(int experts) { return (experts + 1) | 1; }

int sort_warps(int64_t chunk, int experts) {
  int w = kSortThreads / 32;
  while (w > 1 && w * sort_pitch(experts) > kSortSmemWords) w /= 2;
  while (w > 1 && (w / 2) * 32 >= chunk) w /= 2;
  return w;
}

__device__ __forceinline__ int ld_shared_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int key_of(int id, int experts) {
  return (unsigned)id < (unsigned)experts ? id : experts;
}

// Counts per key of one chunk: counts[key * chunks + chunk].
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a, int64_t chunk) {
  extern __shared__ int hist[];
  const int keys = a.experts + 1;
  begin_early(true);
  for (int e = threadIdx.x; e < keys; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * chunk;
  const int64_t end = begin + chunk < a.slots ? begin + chunk : a.slots;
  for (int64_t s = begin + threadIdx.x; s < end; s += blockDim.x)
    atomicAdd(&hist[key_of(a.ids[s], a.experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += blockDim.x)
    a.workspace[(int64_t)e * gridDim.x + blockIdx.x] = hist[e];
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

// Exclusive prefix of one key's counts over the warps, in place; returns their sum.
__device__ __forceinline__ int prefix_over_warps(int* count, int warps, int pitch) {
  int sum = 0;
  for (int w0 = 0; w0 < warps; w0 += 8) {
    int c[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? count[(w0 + w) * pitch] : 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w0 + w < warps) count[(w0 + w) * pitch] = sum;
      sum += c[w];
    }
  }
  return sum;
}

// Writes the rows of a warp's slots lo .. hi-1; `seen` counts its slots of each key.
__device__ __forceinline__ void place_segment(const SortArgs& a, int64_t lo, int64_t hi, int* seen,
                                              const int* base) {
  const int lane = threadIdx.x % 32;
  int next = lo + lane < hi ? a.ids[lo + lane] : 0;
  for (int64_t s0 = lo; s0 < hi; s0 += 32) {
    const int64_t s = s0 + lane;
    const bool live = s < hi;
    const int key = key_of(next, a.experts);
    if (s + 32 < hi) next = a.ids[s + 32];
    const unsigned active = __ballot_sync(0xffffffffu, live);
    if (live) {
      const unsigned peers = __match_any_sync(active, key);
      const int rank = __popc(peers & ((1u << lane) - 1));
      int* h = &seen[key];
      const int place = *h + rank;
      __syncwarp(active);
      if (rank == 0) *h = place + __popc(peers);
      __syncwarp(active);
      const int row = base[key] + place;
      a.row_of_slot[s] = key < a.experts ? row : -1;
      if (a.slot_of_row) a.slot_of_row[row] = key < a.experts ? (int)s : -1;
    }
    __syncwarp();
  }
}

// Rows of one chunk's slots, from the counts of every chunk (at most 32 * LOADS), which one warp
// per key reads side by side.  The ids are read after the wait too, although the counting kernel
// has waited for whoever wrote them: what a kernel wrote is visible to those that wait.
template <int LOADS>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a, int64_t chunk,
                                                                  int warps) {
  extern __shared__ int hist[];  // [warps][pitch], then [keys] first rows and [keys] totals
  __shared__ int warp_sums[32];
  const int keys = a.experts + 1, pitch = sort_pitch(a.experts);
  int* const base = hist + warps * pitch;
  int* const totals = base + keys;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t begin = blockIdx.x * chunk;
  const int64_t end = begin + chunk < a.slots ? begin + chunk : a.slots;
  const int64_t seg = ((end - begin + warps - 1) / warps + 31) / 32 * 32;
  const int64_t lo = begin + warp * seg;
  const int64_t hi = warp < warps ? (lo + seg < end ? lo + seg : end) : lo;

  for (int e = threadIdx.x; e < warps * pitch; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  begin_early(true);
  for (int64_t s = lo + lane; s < hi; s += 32)
    atomicAdd(&hist[warp * pitch + key_of(a.ids[s], a.experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += blockDim.x) prefix_over_warps(hist + e, warps, pitch);

  const int chunks = gridDim.x;
  constexpr int kKeys = 4;  // keys whose counts a warp has in flight
  for (int e0 = warp; e0 < keys; e0 += kKeys * (blockDim.x / 32)) {
    int c[kKeys][LOADS];
#pragma unroll
    for (int n = 0; n < kKeys; ++n) {
      const int e = e0 + n * (blockDim.x / 32);
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        c[n][i] = e < keys && i * 32 + lane < chunks
                      ? a.workspace[(int64_t)e * chunks + i * 32 + lane]
                      : 0;
    }
#pragma unroll
    for (int n = 0; n < kKeys; ++n) {
      const int e = e0 + n * (blockDim.x / 32);
      if (e >= keys) break;
      int all = 0, before = 0;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        all += c[n][i];
        before += i * 32 + lane < (int)blockIdx.x ? c[n][i] : 0;
      }
      all = __reduce_add_sync(0xffffffffu, all);
      before = __reduce_add_sync(0xffffffffu, before);
      if (lane == 0) {
        totals[e] = all;
        base[e] = before;
      }
    }
  }
  __syncthreads();

  int carry = 0;
  for (int e0 = 0; e0 < keys; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int total;
    const int first = carry + block_exclusive(e < keys ? totals[e] : 0, warp_sums, total);
    carry += total;
    if (e < keys) {
      base[e] += first;
      if (blockIdx.x == 0) a.offsets[e] = first;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[keys] = (int)a.slots;
  __syncthreads();

  place_segment(a, lo, hi, hist + warp * pitch, base);
}

// The same in one launch for fewer slots: the chunks' blocks are one cluster (or a single block),
// each adds up its warps' counts, one thread per key, and reads the others' from their shared
// memory.
__global__ void __launch_bounds__(kSortThreads) sort_cluster_kernel(SortArgs a, int64_t chunk,
                                                                    int warps) {
  extern __shared__ int hist[];  // [warps][pitch], [keys] first rows, [keys] this block's counts
  __shared__ int warp_sums[32];
  const int keys = a.experts + 1, pitch = sort_pitch(a.experts);
  int* const base = hist + warps * pitch;
  int* const counts = base + keys;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t begin = blockIdx.x * chunk;
  const int64_t end = begin + chunk < a.slots ? begin + chunk : a.slots;
  const int64_t seg = ((end - begin + warps - 1) / warps + 31) / 32 * 32;
  const int64_t lo = begin + warp * seg;
  const int64_t hi = warp < warps ? (lo + seg < end ? lo + seg : end) : lo;

  for (int e = threadIdx.x; e < warps * pitch; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  begin_early(true);
  for (int64_t s = lo + lane; s < hi; s += 32)
    atomicAdd(&hist[warp * pitch + key_of(a.ids[s], a.experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < keys; e += blockDim.x)
    counts[e] = prefix_over_warps(hist + e, warps, pitch);
  if (gridDim.x > 1) cluster_sync();
  // (block_exclusive's barriers order a single block's counts: each is read by its writer)

  int carry = 0;
  for (int e0 = 0; e0 < keys; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int all = 0, before = 0, total;
    if (e < keys) {
      const uint32_t at = smem_u32(counts + e);
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int c = ld_shared_cluster(mapa_shared(at, b));
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    }
    const int first = carry + block_exclusive(all, warp_sums, total);
    carry += total;
    if (e < keys) {
      base[e] = first + before;
      if (blockIdx.x == 0) a.offsets[e] = first;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[keys] = (int)a.slots;
  __syncthreads();
  place_segment(a, lo, hi, hist + warp * pitch, base);
  if (gridDim.x > 1) cluster_sync();  // no block's counts go away while another reads them
}

// ---------------------------------------------------------------------------------------
// weighted sum of a token's rows, and its gradient
//
// Bound by HBM: every named row of C is read once.  A thread takes 8 columns of a token (16-byte
// accesses, a warp's are 512 bytes of a row) and has the rows of up to 8 slots in flight, as
// many as top_k needs; the registers are held to what leaves 1024 to 2048 threads per SM (the
// gradient's 8 rows 80 registers and 768 threads).
//   sum, 8 rows     blocks of 64 threads, 64 registers: 8192 tokens of 7168 columns 140 us,
//                   6.9 TB/s (70 registers 146, 128 threads 145, 256 threads with 70 172)
//   4 / 2 rows      128 threads: 8192 tokens of 4096 columns 61.4 / 41.5 us (64 threads 61.9 /
//                   41.7; left to itself the compiler took 63.3 us for 4)
//   1 row           128 threads and two vectors of columns per thread, else a block ends before
//                   enough loads are out: 16384 tokens of 4096 columns 45 us (one vector 48, 64
//                   threads 68)
//   gradient        a token's whole row for its dot products, one block of 256 threads, no
//                   partial sums to be joined in memory: 4096 tokens x 8 rows of 7168 columns
//                   149 us, 6.7 TB/s (64 threads 153)
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ int checked_row(const int32_t* row_of_slot, int64_t slot,
                                           int64_t in_rows, int* err) {
  const int row = row_of_slot[slot];
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

// SLOTS rows of a token in flight per thread, each in kCombineVecs vectors of 8 columns.
template <int SLOTS>
constexpr int kCombineThreads = SLOTS == 8 ? 64 : 128;
template <int SLOTS>
constexpr int kCombineBlocks = SLOTS == 4 ? 12 : 16;  // per SM
template <int SLOTS>
constexpr int kCombineVecs = SLOTS == 1 ? 2 : 1;

template <int SLOTS>
__global__ void __launch_bounds__(kCombineThreads<SLOTS>, kCombineBlocks<SLOTS>)
    combine_kernel(CombineArgs a, bool early) {
  constexpr int VECS = kCombineVecs<SLOTS>;
  const int64_t t = blockIdx.x;
  const int first = (blockIdx.y * VECS * blockDim.x + threadIdx.x) * 8;
  const int step = blockDim.x * 8;
  begin_early(early);
  float acc[VECS][8] = {};
  if (a.residual) {
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      uint32_t w[4];
      if (first + v * step < a.N) {
        load_words(static_cast<const uint16_t*>(a.residual) + t * a.N + first + v * step, w);
        unpack8(w, acc[v]);
      }
    }
  }
  for (int j0 = 0; j0 < a.top_k; j0 += SLOTS) {
    uint32_t w[SLOTS][VECS][4];
    int row[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
      row[j] = j0 + j < a.top_k
                   ? checked_row(a.row_of_slot, t * a.top_k + j0 + j, a.in_rows, a.err)
                   : -1;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
#pragma unroll
      for (int v = 0; v < VECS; ++v)
        if (row[j] >= 0 && first + v * step < a.N)
          load_words(static_cast<const uint16_t*>(a.C) + (int64_t)row[j] * a.N + first + v * step,
                     w[j][v]);
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      if (row[j] < 0) continue;
      const float g = a.weights ? a.weights[t * a.top_k + j0 + j] : 1.0f;
#pragma unroll
      for (int v = 0; v < VECS; ++v) {
        float c[8];
        unpack8(w[j][v], c);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[v][e] = fmaf(g, c[e], acc[v][e]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < VECS; ++v)
    if (first + v * step < a.N)
      st_global_v4(static_cast<uint16_t*>(a.out) + t * a.N + first + v * step,
                   pack_bf16x2(acc[v][0], acc[v][1]), pack_bf16x2(acc[v][2], acc[v][3]),
                   pack_bf16x2(acc[v][4], acc[v][5]), pack_bf16x2(acc[v][6], acc[v][7]));
}

template <int SLOTS>
__global__ void __launch_bounds__(256, SLOTS == 8 ? 3 : SLOTS == 4 ? 4 : 6)
    combine_backward_kernel(CombineBackwardArgs a, bool early) {
  __shared__ float part[8][SLOTS];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  begin_early(early);
  for (int j0 = 0; j0 < a.top_k; j0 += SLOTS) {
    int row[SLOTS];
    float g[SLOTS], dot[SLOTS] = {};
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      const bool there = j0 + j < a.top_k;
      row[j] = there ? checked_row(a.row_of_slot, t * a.top_k + j0 + j, a.in_rows, a.err) : -1;
      g[j] = there ? a.weights[t * a.top_k + j0 + j] : 0.0f;
    }
    for (int col = threadIdx.x * 8; col < a.N; col += blockDim.x * 8) {
      uint32_t wd[4], w[SLOTS][4];
      float d[8];
      load_words(static_cast<const uint16_t*>(a.d_out) + t * a.N + col, wd);
#pragma unroll
      for (int j = 0; j < SLOTS; ++j)
        if (row[j] >= 0)
          load_words(static_cast<const uint16_t*>(a.C) + (int64_t)row[j] * a.N + col, w[j]);
      unpack8(wd, d);
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
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
    for (int j = 0; j < SLOTS; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o /= 2) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < SLOTS && j0 + (int)threadIdx.x < a.top_k) {
      float s = 0.0f;
      for (int w = 0; w < (int)blockDim.x / 32; ++w) s += part[w][threadIdx.x];
      a.d_weights[t * a.top_k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// Once per device the kernels are allowed the most that any sort asks for.  What a launch may
// use belongs to the kernel, not to the call: several host threads may sort at once, and no call
// may take away what another is about to launch with.
cudaError_t allow_sort_smem() {
  constexpr size_t kMost = (kSortSmemWords + 2 * (kSortMaxExperts + 1)) * sizeof(int);
  static_assert(kMost + 1024 <= 227 * 1024, "shared memory per block");
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  for (const void* kernel : {reinterpret_cast<const void*>(sort_cluster_kernel),
                             reinterpret_cast<const void*>(sort_place_kernel<2>),
                             reinterpret_cast<const void*>(sort_place_kernel<kSortMaxChunks / 32>)}) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
  }
  if (dev < 64) done[dev].store(true, std::memory_order_release);
  return cudaSuccess;
}

}  // namespace

int64_t moe_sort_workspace_bytes(int64_t slots, int experts) {
  if (slots <= kSortCluster) return 0;
  const int64_t chunk = sort_chunk(slots);
  return (slots + chunk - 1) / chunk * (experts + 1) * (int64_t)sizeof(int32_t);
}

cudaError_t launch_moe_sort(const SortArgs& a, cudaStream_t stream) {
  const int keys = a.experts + 1;
  const int blocks = a.slots <= kSortSingle ? 1 : a.slots <= kSortCluster ? kSortClusterBlocks : 0;
  const int64_t chunk = blocks ? (a.slots + blocks - 1) / blocks : sort_chunk(a.slots);
  const int warps = sort_warps(chunk, a.experts);
  // one thread per key in the scan, as far as a block goes
  int threads = (keys + 31) / 32 * 32;
  threads = threads < warps * 32 ? warps * 32 : threads;
  threads = threads < kSortThreads ? threads : kSortThreads;
  const size_t smem = ((size_t)warps * sort_pitch(a.experts) + 2 * keys) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_sort_smem();
    if (e != cudaSuccess) return e;
  }
  if (blocks)
    return launch(sort_cluster_kernel, blocks, threads, smem, true, stream, blocks, a, chunk, warps);
  const int chunks = (int)((a.slots + chunk - 1) / chunk);
  const auto place = chunks <= 64 ? sort_place_kernel<2> : sort_place_kernel<kSortMaxChunks / 32>;
  const cudaError_t c = launch(sort_count_kernel, chunks, kSortThreads, keys * sizeof(int), true,
                               stream, 1, a, chunk);
  if (c != cudaSuccess) return c;
  // starts, and clears its histograms, while the counts are still being made
  return launch(place, chunks, threads, smem, true, stream, 1, a, chunk, warps);
}

template <int SLOTS>
cudaError_t combine_as(const CombineArgs& a, cudaStream_t stream) {
  constexpr int kMost = kCombineThreads<SLOTS>, kVecs = kCombineVecs<SLOTS>;
  const int pieces = (a.N / 8 + kVecs - 1) / kVecs;  // threads to a row
  const int parts = (pieces + kMost - 1) / kMost;    // blocks to a row
  const int threads = ((pieces + parts - 1) / parts + 31) / 32 * 32;
  const dim3 grid((unsigned)a.rows, (unsigned)parts);
  const bool early =
      starts_early(grid, (int64_t)threads * kVecs * 16 * (a.top_k + 1 + (a.residual ? 1 : 0)));
  return launch(combine_kernel<SLOTS>, grid, threads, 0, early, stream, 1, a, early);
}

cudaError_t launch_moe_combine(const CombineArgs& a, cudaStream_t stream) {
  return a.top_k <= 1   ? combine_as<1>(a, stream)
         : a.top_k <= 2 ? combine_as<2>(a, stream)
         : a.top_k <= 4 ? combine_as<4>(a, stream)
                        : combine_as<8>(a, stream);
}

cudaError_t launch_moe_combine_backward(const CombineBackwardArgs& a, cudaStream_t stream) {
  const int vecs = a.N / 8;
  const int threads = vecs >= 256 ? 256 : (vecs + 31) / 32 * 32;
  const auto kernel = a.top_k <= 2   ? combine_backward_kernel<2>
                      : a.top_k <= 4 ? combine_backward_kernel<4>
                                     : combine_backward_kernel<8>;
  const bool early = starts_early((unsigned)a.rows, (int64_t)a.N * 2 * (2 * a.top_k + 1));
  return launch(kernel, (unsigned)a.rows, threads, 0, early, stream, 1, a, early);
}

}  // namespace bsfp8
