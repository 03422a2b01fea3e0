// Quantisation along the rows, the operands of the 8-bit weight gradient: in every group, blocks of
// 128 rows of a column counted from the group's first row,
//
//   a = largest |x| of the block,  scale = a / 448 (at least 2^-126; 1 for zeros; NaN where the
//   block holds a NaN or an infinity),  q = e4m3(x / scale)
//
// the blockwise rule of quant.cuh turned by 90 degrees.  Rows may be gathered: row r of q comes
// from the token whose slot lies in row r.  Each element is read once, kept in registers while its
// block's largest magnitude is found, and written once: 65536 rows of 7168 take 216 us, 6.6 TB/s,
// what HBM gives.  Gathered from 8192 tokens the same rows come out of L2, and at 169 us
// instructions and barriers bound it (with the loads left out 147).
//
// A block of threads takes the 128 rows of a scale block and walks over tiles of 128 or 64 columns, the
// next ones under way (cp.async; a thread reads back what it copied itself): thread (i, c) the 8
// columns 8 c.. of the rows i, i + 16, .., so that 16 (8) threads read 256 (128) bytes of a row
// (16-bit) and write half as many.  Which rows those are the offsets say: block b of the scales belongs
// to the last group e with offsets[e] / 128 + e <= b, which the threads count together, once for all
// tiles; the first block reports offsets that are no partition.
#include <cuda_fp16.h>

#include "expert_ops.cuh"
#include "moe_ops.cuh"
#include "quant.cuh"

namespace bsfp8 {
namespace {

constexpr int kBlockRows = 128;
constexpr int kRowThreads = 16;                      // of a column of threads
constexpr int kRowsEach = kBlockRows / kRowThreads;  // 8

template <int XT>
constexpr int kEightBytes = XT == E_FP32 ? 32 : 16;  // of 8 elements as they are stored

// Columns of a tile, tiles in flight and blocks per SM.  16-bit rows that lie side by side come from
// HBM and want long pieces and depth (65536 rows of 7168: 216 us, in tiles of 64 columns 242).  Gathered
// rows come out of L2, and more blocks, whose barriers hold fewer threads, are worth more than more
// tiles: of 8 of 8192 tokens 169 us (128 columns 172, with three tiles 195), 16384 rows by 8 of 2048
// tokens 50 (58).  fp32 fills shared memory with twice the bytes: 16384 rows of 4096 61 us, 77 with
// 128 columns.
template <int XT, bool GATHER>
struct Tile {
  static constexpr int COLS = GATHER || XT == E_FP32 ? 64 : 128;
  static constexpr int COLUMN_THREADS = COLS / 8;  // side by side
  static constexpr int THREADS = kRowThreads * COLUMN_THREADS;
  static constexpr int STAGES = GATHER ? 2 : 3;
  static constexpr int RESIDENT = XT == E_FP32 ? 2 : GATHER ? 6 : 2;
  static constexpr int STAGE_BYTES = kBlockRows * COLUMN_THREADS * kEightBytes<XT>;
};

// Eight elements as they are stored.
template <int XT>
struct Eight {
  uint32_t w[kEightBytes<XT> / 4];
};

template <int XT>
__device__ __forceinline__ Eight<XT> read8(const uint8_t* p) {
  Eight<XT> x;
#pragma unroll
  for (int i = 0; i < kEightBytes<XT> / 16; ++i) {
    const uint4 w = reinterpret_cast<const uint4*>(p)[i];
    x.w[4 * i] = w.x;
    x.w[4 * i + 1] = w.y;
    x.w[4 * i + 2] = w.z;
    x.w[4 * i + 3] = w.w;
  }
  return x;
}

// Largest magnitudes of eight columns so far.  16-bit values are compared as they lie: without
// their signs they are ordered as integers, infinities and NaNs last, two to an instruction.
template <int XT>
__device__ __forceinline__ void take_max(Eight<XT>& top, const Eight<XT>& a, const Eight<XT>& b) {
#pragma unroll
  for (int i = 0; i < kEightBytes<XT> / 4; ++i) {
    if constexpr (XT == E_FP32)
      top.w[i] = max(max(top.w[i], a.w[i] & 0x7fffffffu), b.w[i] & 0x7fffffffu);
    else
      top.w[i] = __vimax3_u16x2(top.w[i], a.w[i] & 0x7fff7fffu, b.w[i] & 0x7fff7fffu);
  }
}

template <int XT>
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
  return XT == E_FP32 ? max(a, b) : __vmaxu2(a, b);
}

// The two columns of a word (fp32: one, in v.x).
template <int XT>
__device__ __forceinline__ float2 word_values(uint32_t w) {
  if constexpr (XT == E_FP32) {
    return make_float2(__uint_as_float(w), 0.0f);
  } else if constexpr (XT == E_BF16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

// Elements 2 j and 2 j + 1.
template <int XT>
__device__ __forceinline__ float2 pair(const Eight<XT>& x, int j) {
  if constexpr (XT == E_FP32)
    return make_float2(__uint_as_float(x.w[2 * j]), __uint_as_float(x.w[2 * j + 1]));
  else
    return word_values<XT>(x.w[j]);
}

template <int XT, bool GATHER>
__global__ void __launch_bounds__(Tile<XT, GATHER>::THREADS, Tile<XT, GATHER>::RESIDENT)
    columns_kernel(ColumnsArgs a, int blocks, int each) {
  extern __shared__ __align__(16) uint8_t stages[];
  using T = Tile<XT, GATHER>;
  constexpr int STAGES = T::STAGES, kTileCols = T::COLS, kThreads = T::THREADS;
  constexpr int kColumnThreads = T::COLUMN_THREADS;
  constexpr int kWords = kEightBytes<XT> / 4;          // of a thread's eight columns
  constexpr int kTileWords = kWords * kColumnThreads;  // of a tile's row
  __shared__ __align__(16) uint32_t part[2][kThreads / 32][kTileWords];
  __shared__ __align__(16) float inverse[2][kTileCols];
  __shared__ int counts[kThreads / 32];
  const int stripe = blockIdx.x / blocks, b = blockIdx.x - stripe * blocks;
  begin_early(true);  // its blocks move 24 KB and more
  // the groups whose first block is b or before it; a group's first block grows with the group
  int before = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const int lo = a.offsets[e], hi = a.offsets[e + 1];
    before += lo / kBlockRows + e <= b;
    const bool good = lo >= 0 && lo <= hi && hi <= a.M_total && (e > 0 || lo == 0);
    if (!good && blockIdx.x == 0) atomicCAS(a.err, 0, (int)DEV_BAD_OFFSETS);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) before += __shfl_xor_sync(0xffffffffu, before, d);
  if (threadIdx.x % 32 == 0) counts[threadIdx.x / 32] = before;
  __syncthreads();
  int e = -1;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) e += counts[i];
  if (e < 0) return;
  const int64_t r0 = a.offsets[e], r1 = a.offsets[e + 1];
  const int64_t first = r0 + (b - (r0 / kBlockRows + e)) * (int64_t)kBlockRows;
  // a block that no group has, or offsets that are no partition (recorded above)
  if (r0 < 0 || r1 > a.M_total || first < r0 || first >= r1) return;
  const int rows = r1 - first < kBlockRows ? (int)(r1 - first) : kBlockRows;

  const int c = threadIdx.x % kColumnThreads, i0 = threadIdx.x / kColumnThreads;
  constexpr int kBytes = XT == E_FP32 ? 4 : 2;
  const int tile0 = stripe * each;
  const int tiles = min(each, a.K / kTileCols - tile0);
  // the rows' elements of the tile that is fetched next; rows that hold nothing are filled with
  // zeros and read nothing (16 bytes or none)
  const char* from[kRowsEach];
  uint32_t bytes[kRowsEach];
#pragma unroll
  for (int j = 0; j < kRowsEach; ++j) {
    const int i = i0 + j * kRowThreads;
    int64_t row = -1;
    if (i < rows) {
      row = first + i;
      if constexpr (GATHER) {
        const int slot = a.slot_of_row[row];
        row = slot < 0 ? -1 : slot / a.top_k;
        if (row >= a.x_rows) {
          atomicCAS(a.err, 0, DEV_BAD_ROWS);
          row = -1;
        }
      }
    }
    bytes[j] = row < 0 ? 0 : 16;
    // (an address for none: x may be NULL where it has no rows)
    from[j] = row < 0 ? reinterpret_cast<const char*>(a.q)
                      : static_cast<const char*>(a.x) + (row * a.K + tile0 * kTileCols + 8 * c) * kBytes;
  }
  uint8_t* const mine = stages + threadIdx.x * kEightBytes<XT>;  // + stage, + row j
  const uint32_t mine_u32 = smem_u32(mine);
  auto fetch = [&](bool any, int stage) {
    if (any) {
      const uint32_t dst = mine_u32 + stage * T::STAGE_BYTES;
#pragma unroll
      for (int j = 0; j < kRowsEach; ++j) {
#pragma unroll
        for (int h = 0; h < kEightBytes<XT>; h += 16)
          cp_async_16(dst + j * kThreads * kEightBytes<XT> + h, from[j] + h, bytes[j]);
        from[j] += kTileCols * kBytes;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s < tiles, s);
  const uint64_t pol = l2_policy_evict_first();  // x is what is read again, by other slots
  uint8_t* q = a.q + (first + i0) * a.K + tile0 * kTileCols + 8 * c;
  float* scale_at = a.scales + (int64_t)b * a.K + tile0 * kTileCols;
  const int64_t q_rows = (int64_t)kRowThreads * a.K;
  const bool full = rows == kBlockRows;
  int stage = 0, side = 0;
  for (int tile = 0; tile < tiles; ++tile, side ^= 1, q += kTileCols, scale_at += kTileCols) {
    fetch(tile + STAGES - 1 < tiles, stage == 0 ? STAGES - 1 : stage - 1);
    cp_async_wait_group<STAGES - 1>();
    Eight<XT> x[kRowsEach], top = {};
#pragma unroll
    for (int j = 0; j < kRowsEach; ++j)
      x[j] = read8<XT>(mine + stage * T::STAGE_BYTES + j * kThreads * kEightBytes<XT>);
    if (++stage == STAGES) stage = 0;
#pragma unroll
    for (int j = 0; j < kRowsEach; j += 2) take_max<XT>(top, x[j], x[j + 1]);
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int d = 16; d >= kColumnThreads; d /= 2)
        top.w[i] = max_words<XT>(top.w[i], __shfl_xor_sync(0xffffffffu, top.w[i], d));
    if (threadIdx.x % 32 < kColumnThreads) {
      uint4* p = reinterpret_cast<uint4*>(&part[side][threadIdx.x / 32][kWords * c]);
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        p[i] = make_uint4(top.w[4 * i], top.w[4 * i + 1], top.w[4 * i + 2], top.w[4 * i + 3]);
    }
    __syncthreads();
    if (threadIdx.x < kTileWords) {  // a word's columns each: their scales and those's reciprocals
      uint32_t m = part[side][0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < kThreads / 32; ++w) m = max_words<XT>(m, part[side][w][threadIdx.x]);
      const float2 amax = word_values<XT>(m);
      constexpr int kCols = XT == E_FP32 ? 1 : 2;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const float a_i = i ? amax.y : amax.x;
        const int col = threadIdx.x * kCols + i;
        const bool finite = a_i < __int_as_float(0x7f800000);
        const float scale = a_i == 0.0f ? 1.0f : fmaxf(__fdiv_rn(a_i, 448.0f), 0x1p-126f);
        scale_at[col] = finite ? scale : __int_as_float(0x7fffffff);
        inverse[side][col] = finite ? __frcp_rn(scale) : 0.0f;
      }
    }
    __syncthreads();
    const float4 lo = *reinterpret_cast<const float4*>(&inverse[side][8 * c]);
    const float4 hi = *reinterpret_cast<const float4*>(&inverse[side][8 * c + 4]);
    const float2 inv[4] = {{lo.x, lo.y}, {lo.z, lo.w}, {hi.x, hi.y}, {hi.z, hi.w}};
    auto store = [&](int j, uint8_t* to) {
      uint32_t code[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 v = pair<XT>(x[j], i);
        mul2(v.x, v.y, inv[i].x, inv[i].y, v.x, v.y);
        code[i] = cvt_e4m3x2(v.x, v.y);
      }
      st_global_v2_hint(to, code[0] | (code[1] << 16), code[2] | (code[3] << 16), pol);
    };
    uint8_t* to = q;
    if (full) {
#pragma unroll
      for (int j = 0; j < kRowsEach; ++j, to += q_rows) store(j, to);
    } else {
#pragma unroll
      for (int j = 0; j < kRowsEach; ++j, to += q_rows)
        if (i0 + j * kRowThreads < rows) store(j, to);
    }
  }
}

template <int XT, bool GATHER>
cudaError_t columns_as(const ColumnsArgs& a, cudaStream_t stream) {
  // A stripe of columns for all row blocks, then the next: what is gathered several times stays in
  // L2 that long.  A block's way to its rows (offsets, slots, rows) is three round trips to L2, so
  // stripes are no narrower than it takes to keep the SMs busy to the end (to the end of little work: 900
  // blocks, 32896 gathered rows of 512 17.0 -> 14.6 us, 6000 rows of 2176 in 60 groups 13.2 -> 10.1).
  using T = Tile<XT, GATHER>;
  constexpr int kSmem = T::STAGES * T::STAGE_BYTES;
  const cudaError_t e = allow_smem<columns_kernel<XT, GATHER>>(kSmem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = a.M_total / kBlockRows + a.E;
  const int tiles = a.K / T::COLS;
  const int64_t most = blocks * tiles < 8000 ? 900 : 2500, want = (most + blocks - 1) / blocks;
  const int each = (int)((tiles + want - 1) / want);
  const dim3 grid((unsigned)(blocks * ((tiles + each - 1) / each)));
  return launch(columns_kernel<XT, GATHER>, grid, T::THREADS, kSmem, true, stream, 1, a, (int)blocks, each);
}

}  // namespace

cudaError_t launch_quantize_columns(int x_type, const ColumnsArgs& a, cudaStream_t stream) {
  const bool gather = a.slot_of_row != nullptr;
  switch (x_type) {
    case E_BF16: return gather ? columns_as<E_BF16, true>(a, stream) : columns_as<E_BF16, false>(a, stream);
    case E_FP16: return gather ? columns_as<E_FP16, true>(a, stream) : columns_as<E_FP16, false>(a, stream);
    default: return gather ? columns_as<E_FP32, true>(a, stream) : columns_as<E_FP32, false>(a, stream);
  }
}

}  // namespace bsfp8
