// Matrix products grouped by expert in bf16 or fp16 for sm_103a (persistent, warp specialised):
//
//   C[m, n] = sum_k A[m, k] * B[e, n, k]        e the expert of row m's group
//   C[m, n] = sum_k A[m, k] * B[e, k, n]        transposed: the gradient of the product's rows
//
// fp32 accumulation in TMEM, each result rounded once.  Both forms read the weights as they lie:
// a tile of B[e, n, k] is a K-major operand of the MMA, one of B[e, k, n] an MN-major one.  The
// weights are mapped as a stack of matrices, so that a tile past an expert's last row or column
// reads zeros and not the next expert; rows of A past a group's end belong to its neighbour, give
// rows of the tile that are not stored, and touch no others.
//
// Two kernels, for what bounds them:
//   few rows per expert: the weights' bytes.  One CTA takes 32 rows x 128 columns, and what counts is
//   how many bytes are in flight: 9 stages of 16 KB of weights per SM.  The MMA (M = 128 rows of A)
//   computes 96 rows that nobody reads.  512 rows over 128 experts of 4096 x 2048: 307 us, 7.0 TB/s,
//   more than a copy's rate, as next to nothing is written.  Where the tiles are fewer than the SMs,
//   clusters of CTAs share a tile's K and add up their parts through distributed shared memory.
//   more rows: the tensor core, and the way from L2 to it.  A CTA pair takes 256 columns x up to 512
//   rows; the rows are the MMA's N, which goes by 16, so that a group's last rows cost what they are.
//   8192^3: 563 us, 1950 TFLOP/s (a library product 557).
//   8 groups of 512 rows, 4096 x 7168: 153 us, the tensor cores busy 90 % of the time that the SMs
//   are; uneven groups of 4096 rows in long runs, under the power cap, 181.
// In both: a TMA producer, an MMA thread (per 64 K four MMAs of K = 16 and one commit) and epilogue
// warps that store one tile while the next accumulates in the other half of TMEM.
#include "expert_ops.cuh"
#include "operand_ring.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace bsfp8 {
namespace g16 {

constexpr int BK = 64;  // elements: 128 bytes

// The tensor core's additions truncate: a sum of n terms of one sign in one accumulator comes out
// 6.4e-9 n of it short.  So an accumulator takes parts of K of at most 16384 for fp16 results (1.05e-4 of
// the sum, less than half of a rounding, which is 2.4e-4 to 4.9e-4) and 131072 for bf16 (8.4e-4; 2.0e-3 to
// 3.9e-3), and longer parts are summed in chunks of 4096 that are added up in fp32 (2.6e-5 whatever K is;
// in one accumulator a K of 2^20 lost 6.7e-3).  Chunks want a thread's sums in registers, in tiles of up to
// 256 rows: 8192 x 8192 x 65536 in fp16 5.1-5.4 ms, in one accumulator 4.8.
constexpr int MOST_BLOCKS_FP16 = 16384 / BK, MOST_BLOCKS_BF16 = 131072 / BK;
constexpr int CHUNK_BLOCKS = 4096 / BK;

// The tiles that CTA (or pair) `unit` of `units` takes: one of every `units`, in each round the next
// place.  Row tiles of a group follow one another in the numbering, the last often a small one; at
// a fixed place some units would get all the full ones (64 groups of 70 to 900 rows, 7168 x 2048:
// 167 us, in turns 159).
struct Turns {
  int64_t at, round;
  uint32_t place;
  const uint32_t units;
  __device__ Turns(int64_t unit, int64_t units_)
      : at(unit), round(0), place((uint32_t)unit), units((uint32_t)units_) {}
  __device__ void next() {
    round += units;
    if (++place == units) place = 0;
    at = round + place;
  }
};

// The groups that have rows, in shared memory: the first row and the expert of each, and behind them
// the last one's end.  A walk over the offsets themselves waits for L2 at every group, empty ones too
// (9 rows in 128 groups, 168 x 864: 17.9 us, listed 6.2).  Above LISTED of them the walk does that.
constexpr int LISTED = 128;
struct GroupList {
  int count;  // or -1: too many
  int2 at[LISTED + 1];
};

// One full warp lists the groups, checks them (as check_offsets does, and the expert ids) and counts
// their tiles of BM rows.
template <int BM>
__device__ __forceinline__ int list_groups(const Product16Args& a, GroupList& list, int64_t& row_tiles) {
  constexpr int kAhead = 4;  // loads of 32 groups each, under way together
  const uint32_t lane = lane_id();
  int good = 1, good_ids = 1, count = 0;
  long long tiles = 0;
  for (int e0 = 0; e0 < a.E; e0 += 32 * kAhead) {
    int lo[kAhead], hi[kAhead], be[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int e = e0 + 32 * i + (int)lane;
      const bool in = e < a.E;
      lo[i] = in ? a.offsets[e] : 0;
      hi[i] = in ? a.offsets[e + 1] : 0;
      be[i] = in && a.expert_ids ? a.expert_ids[e] : e;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int e = e0 + 32 * i + (int)lane;
      if (lo[i] < 0 || hi[i] < lo[i] || hi[i] > a.M_total || (e == 0 && lo[i] != 0)) good = 0;
      if (e < a.E && (be[i] < 0 || be[i] >= a.num_experts)) good_ids = 0;
      const bool some = hi[i] > lo[i];
      if (some) tiles += ((int64_t)hi[i] - lo[i] + BM - 1) / BM;
      const uint32_t others = __ballot_sync(0xffffffffu, some);
      const int at = count + __popc(others & ((1u << lane) - 1));
      if (some && at < LISTED) list.at[at] = make_int2(lo[i], be[i]);
      count += __popc(others);
    }
  }
  for (int s = 16; s > 0; s >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, s);
  row_tiles = tiles;
  if (lane == 0) {
    list.count = count <= LISTED ? count : -1;
    list.at[count < LISTED ? count : LISTED] = make_int2(a.offsets[a.E], 0);
  }
  return !__all_sync(0xffffffffu, good)       ? DEV_BAD_OFFSETS
         : !__all_sync(0xffffffffu, good_ids) ? DEV_BAD_EXPERT_IDS
                                              : 0;
}

// The tiles, group by group, of BM rows x BN columns; in a group by bands of BAND row tiles, in a
// band column by column (sched.cuh's order).
template <int BM, int BN, int BAND>
struct GroupWalk {
  int g = -1, be = 0;
  int64_t base = 0, tiles = 0;  // the first tile of group g, and how many it has
  int r0 = 0, r1 = 0;

  // t must not decrease between calls.  Returns false past the last tile.
  __device__ bool locate(const Product16Args& a, const GroupList& list, int64_t t, TileCoord& c) {
    const int nt = (a.N + BN - 1) / BN;  // the last column tile may be partial
    const bool listed = list.count >= 0;
    while (t >= base + tiles) {
      base += tiles;
      ++g;
      if (g >= (listed ? list.count : a.E)) return false;
      if (listed) {
        const int2 at = list.at[g];
        r0 = at.x;
        be = at.y;
        r1 = list.at[g + 1].x;
      } else {
        r0 = a.offsets[g];
        r1 = a.offsets[g + 1];
        be = a.expert_ids ? a.expert_ids[g] : g;
      }
      tiles = ((int64_t)r1 - r0 + BM - 1) / BM * nt;
    }
    c.e = g;
    c.be = be;
    c.m_end = r1;
    const uint32_t rows = (uint32_t)(((int64_t)r1 - r0 + BM - 1) / BM);
    if (tiles <= UINT32_MAX) {  // divisions in 64 bits take half a microsecond
      const uint32_t local = (uint32_t)(t - base);
      const uint32_t band = local / (BAND * (uint32_t)nt), in_band = local - band * (BAND * (uint32_t)nt);
      const uint32_t band_rows = rows - band * BAND < BAND ? rows - band * BAND : BAND;
      const uint32_t col = in_band / band_rows;
      c.m0 = r0 + (int64_t)(band * BAND + (in_band - col * band_rows)) * BM;
      c.n0 = (int)(col * BN);
    } else {
      const int64_t local = t - base;
      const int64_t band = local / ((int64_t)BAND * nt), in_band = local - band * BAND * nt;
      const int64_t band_rows = rows - band * BAND < BAND ? rows - band * BAND : BAND;
      c.m0 = r0 + (band * BAND + in_band % band_rows) * BM;
      c.n0 = (int)(in_band / band_rows) * BN;
    }
    if constexpr (BSFP8_DEBUG) {
      const bool inside = c.m0 >= r0 && c.m0 < r1 && r1 <= a.M_total && c.n0 >= 0 && c.n0 < a.N &&
                          c.be >= 0 && c.be < a.num_experts;
      if (!inside) {
        atomicCAS(a.err, 0, (int)DEV_BOUNDS);
        return false;
      }
    }
    return true;
  }
};

// ---------------------------------------------------------------------------------------
// Few rows: 32 rows x 128 columns per CTA, or per cluster of SPLIT CTAs that share its K
// ---------------------------------------------------------------------------------------
template <bool BT_, int SPLIT_>
struct Few {
  static constexpr bool BT = BT_;        // B [E, K, N]
  static constexpr int SPLIT = SPLIT_;
};
constexpr int FEW_THREADS = 192;  // warp 0 producer, 1 MMA thread, 4 epilogue (TMEM lanes 0..31)
constexpr int FEW_ROWS = 32, FEW_COLS = 128, FEW_STAGES = 9;
constexpr uint32_t FEW_A = FEW_ROWS * BK * 2, FEW_B = FEW_COLS * BK * 2;
constexpr uint32_t FEW_SMEM_B = FEW_STAGES * FEW_A;
constexpr uint32_t FEW_CTL = FEW_SMEM_B + FEW_STAGES * FEW_B;
// what the MMA reads past the 32 rows of the last stage is B's
static_assert((128 - FEW_ROWS) * BK * 2 <= FEW_STAGES * FEW_B, "A's overhang");
// a split tile's part of the sums, in the ring (which is done with by then): padded rows
constexpr int PART_STRIDE = FEW_COLS + 4;
static_assert(FEW_ROWS * PART_STRIDE * 4 <= FEW_CTL, "part");

struct FewCtl {
  uint64_t full[FEW_STAGES];
  uint64_t empty[FEW_STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  long long total_tiles;
  TileCoord tile;  // that a cluster shares
  GroupList list;
};
constexpr uint32_t kFewSmem = FEW_CTL + sizeof(FewCtl) + 1024;  // + alignment slack

__device__ __forceinline__ float4 load_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <class F>
__global__ void __launch_bounds__(FEW_THREADS, 1)
product16_few_kernel(const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmB, const Product16Args args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  FewCtl* ctl = reinterpret_cast<FewCtl*>(smem + FEW_CTL);
  volatile int* abort = &ctl->abort;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t part = F::SPLIT > 1 ? cluster_ctarank() : 0;
  const int KB = (args.K + BK - 1) / BK;
  const int kb0 = (int)((int64_t)KB * part / F::SPLIT);
  const int kb1 = (int)((int64_t)KB * (part + 1) / F::SPLIT);
  const int64_t tile0 = blockIdx.x / F::SPLIT;
  const int64_t tile_stride = gridDim.x / F::SPLIT;

  const uint32_t sA = smem_u32(smem), sB = smem_u32(smem + FEW_SMEM_B);
  auto full_bar = [&](int s) { return smem_u32(&ctl->full[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&ctl->empty[s]); };
  auto tfull_bar = [&](int s) { return smem_u32(&ctl->tfull[s]); };
  auto tempty_bar = [&](int s) { return smem_u32(&ctl->tempty[s]); };
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    for (int s = 0; s < FEW_STAGES; ++s) {
      mbar_init(full_bar(s), 1);   // the producer (+ bytes)
      mbar_init(empty_bar(s), 1);  // one commit
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull_bar(s), 1);   // one commit
      mbar_init(tempty_bar(s), 1);  // the epilogue warp
    }
    mbar_init(smem_u32(&ctl->mma_done), 1);
    ctl->abort = 0;
    ctl->tile = TileCoord{};
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(&ctl->tmem_base), 2 * FEW_COLS);
    tmem_relinquish<1>();
    launch_dependents();
  }
  wait_for_previous();
  if (warp == 2) {
    int64_t row_tiles;
    const int status = list_groups<FEW_ROWS>(args, ctl->list, row_tiles);
    if (lane == 0) {
      ctl->total_tiles = status ? 0 : row_tiles * ((args.N + FEW_COLS - 1) / FEW_COLS);
      if (status && blockIdx.x == 0) atomicCAS(args.err, 0, status);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const int64_t total_tiles = ctl->total_tiles;

  GroupWalk<FEW_ROWS, FEW_COLS, 1> sched;
  TileCoord tc;
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------- TMA producer -------------------------------
      const uint64_t pol_a = l2_policy_evict_last(), pol_b = l2_policy_evict_first();
      uint32_t stage = 0, phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (Turns t(tile0, tile_stride); ok && t.at < total_tiles; t.next()) {
        if (!sched.locate(args, ctl->list, t.at, tc)) break;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_sleep(empty_bar(stage), phase ^ 1, abort)) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          const uint32_t a = sA + stage * FEW_A, b = sB + stage * FEW_B, bar = full_bar(stage);
          mbar_arrive_expect_tx(bar, FEW_A + FEW_B);
          if constexpr (F::BT) {
            tma_load_3d_hint(b, &tmB, tc.n0, kb * BK, tc.be, bar, pol_b);
            tma_load_3d_hint(b + FEW_B / 2, &tmB, tc.n0 + 64, kb * BK, tc.be, bar, pol_b);
          } else {
            tma_load_3d_hint(b, &tmB, kb * BK, tc.n0, tc.be, bar, pol_b);
          }
          tma_load_2d_hint(a, &tmA, kb * BK, (int32_t)tc.m0, bar, pol_a);
          ++issued;
          if (++stage == FEW_STAGES) { stage = 0; phase ^= 1; }
        }
      }
      // the last loads land, and the MMAs that read them end, before the CTA can exit (after an
      // abort the first wait runs out, which is time enough for the loads)
      const int64_t pending = issued < FEW_STAGES ? issued : FEW_STAGES;
      for (int64_t i = 0; i < pending; ++i) {
        stage = (stage + FEW_STAGES - 1) % FEW_STAGES;
        if (stage == FEW_STAGES - 1) phase ^= 1;
        if (!mbar_wait_timed(empty_bar(stage), phase)) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // -------------------------------- MMA thread --------------------------------
      const uint32_t idesc = idesc_f16_f32(128, FEW_COLS) | (F::BT ? IDESC_B_MN : 0u) |
                             (args.bf16 ? IDESC_BF16 : 0u);
      const uint64_t adesc0 = kmajor_sw128_desc(sA);
      const uint64_t bdesc0 = F::BT ? mnmajor_sw128_desc(sB, FEW_B / 2) : kmajor_sw128_desc(sB);
      // 16 K: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major box
      constexpr uint64_t kStepA = 32 >> 4, kStepB = (F::BT ? 2048 : 32) >> 4;
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      for (Turns t(tile0, tile_stride); ok && t.at < total_tiles; t.next()) {
        if (!sched.locate(args, ctl->list, t.at, tc)) break;
        ok = mbar_wait_sleep(tempty_bar(acc), acc_phase ^ 1, abort);
        const uint32_t d = tmem_base + acc * FEW_COLS;
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          ok = mbar_wait_sleep(full_bar(stage), phase, abort);
          if (!ok) break;
          tc_fence_after();
          const uint64_t adesc = adesc0 + ((stage * FEW_A) >> 4);
          const uint64_t bdesc = bdesc0 + ((stage * FEW_B) >> 4);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_f16<1>(d, adesc + k * kStepA, bdesc + k * kStepB, idesc, kb > kb0 || k > 0);
          umma_commit(empty_bar(stage));
          if (++stage == FEW_STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) {
          give_up(args.err, abort);
          break;
        }
        umma_commit(tfull_bar(acc));
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      // every MMA has finished before TMEM is released
      umma_commit(smem_u32(&ctl->mma_done));
      if (!mbar_wait_timed(smem_u32(&ctl->mma_done), 0)) give_up(args.err, abort);
    }
    __syncwarp();
  } else if (warp == 4) {
    // --------------------------------- epilogue ---------------------------------
    uint16_t* Cmat = static_cast<uint16_t*>(args.C);
    const bool wide = (reinterpret_cast<uintptr_t>(args.C) & 31) == 0 && args.N % 16 == 0;
    const uint64_t pol_c = l2_policy_evict_first();
    uint32_t acc = 0, acc_phase = 0;
    for (Turns t(tile0, tile_stride); t.at < total_tiles; t.next()) {
      if (!sched.locate(args, ctl->list, t.at, tc)) break;
      const int64_t row = tc.m0 + lane;
      if (F::SPLIT > 1 && lane == 0) ctl->tile = tc;
      if (!__all_sync(0xffffffffu, mbar_wait_sleep(tfull_bar(acc), acc_phase, abort))) {
        if (lane == 0) give_up(args.err, abort);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + acc * FEW_COLS;
      uint16_t* dst = Cmat + row * (int64_t)args.N + tc.n0;
      const int cols = args.N - tc.n0;  // that are left of the matrix
#pragma unroll 1
      for (int c = 0; c < FEW_COLS; c += 32) {
        uint32_t p[32];
        tmem_ld_32x32b_x32(taddr + c, p);
        tmem_ld_wait();
        if constexpr (F::SPLIT > 1) {
          if (row >= tc.m_end) continue;
          uint4* to = reinterpret_cast<uint4*>(smem + (lane * PART_STRIDE + c) * 4);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            to[j] = make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
        } else {
          if (c + 32 == FEW_COLS) {  // TMEM is read: the MMA thread may have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(acc));
          }
          if (row >= tc.m_end) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float lo = __uint_as_float(p[16 * h + 2 * j]);
              const float hi = __uint_as_float(p[16 * h + 2 * j + 1]);
              v[j] = args.bf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
            }
            const int at = c + 16 * h;
            if (wide) {
              if (at < cols) st_global_v8_hint(dst + at, v, pol_c);
            } else {  // N is a multiple of 8
              if (at < cols) st_global_v4_hint(dst + at, v[0], v[1], v[2], v[3], pol_c);
              if (at + 8 < cols) st_global_v4_hint(dst + at + 8, v[4], v[5], v[6], v[7], pol_c);
            }
          }
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  }

  if constexpr (F::SPLIT > 1) {
    // The parts of the one tile that the cluster has: each CTA adds up a stripe of its columns, in
    // the CTAs' order.  (A CTA that gave up has said so, and the sums mean nothing.)
    cluster_sync();
    if (tile0 < total_tiles) {
      tc = ctl->tile;
      constexpr int kCols = FEW_COLS / F::SPLIT, kGroups = kCols / 4;
      const uint32_t mine = smem_u32(smem);
      for (int i = threadIdx.x; i < FEW_ROWS * kGroups; i += FEW_THREADS) {
        const int r = i / kGroups, c = (int)part * kCols + i % kGroups * 4;
        const int64_t row = tc.m0 + r;
        const int n = tc.n0 + c;
        if (row >= tc.m_end || n >= args.N) continue;  // N is a multiple of 8
        float4 v[F::SPLIT];
#pragma unroll
        for (int s = 0; s < F::SPLIT; ++s)
          v[s] = load_cluster_f4(mapa_shared(mine + (r * PART_STRIDE + c) * 4, s));
#pragma unroll
        for (int s = 1; s < F::SPLIT; ++s) {
          v[0].x += v[s].x;
          v[0].y += v[s].y;
          v[0].z += v[s].z;
          v[0].w += v[s].w;
        }
        uint2 w;
        w.x = args.bf16 ? pack_bf16x2(v[0].x, v[0].y) : pack_f16x2(v[0].x, v[0].y);
        w.y = args.bf16 ? pack_bf16x2(v[0].z, v[0].w) : pack_f16x2(v[0].z, v[0].w);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(args.C) + row * (int64_t)args.N + n) = w;
      }
    }
    cluster_sync();  // the parts are read before any of them goes
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem_base, 2 * FEW_COLS);
  }
}

// More tiles than this there are not (the offsets live on the device): full ones and one of each
// group's last rows.
inline int64_t most_tiles(const Product16Args& a, int rows, int cols) {
  const int64_t most_last = a.M_total < a.E ? a.M_total : a.E;
  return (a.M_total / rows + most_last) * (((int64_t)a.N + cols - 1) / cols);
}

template <class F>
cudaError_t launch_few(const Product16Args& args, int64_t max_tiles, int num_sms,
                       cudaStream_t stream) {
  static_assert(kFewSmem <= 227 * 1024, "shared memory per CTA");
  CUtensorMap tmA, tmB;
  const uint64_t a_dims[2] = {(uint64_t)args.K, (uint64_t)args.M_total};
  const uint64_t b_dims[3] = {(uint64_t)(F::BT ? args.N : args.K),
                              (uint64_t)(F::BT ? args.K : args.N), (uint64_t)args.num_experts};
  if (!encode_swizzled(&tmA, 2, args.A, 2, a_dims, FEW_ROWS) ||
      !encode_swizzled(&tmB, 2, args.B, 3, b_dims, F::BT ? BK : FEW_COLS))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<product16_few_kernel<F>>(kFewSmem);
  if (e != cudaSuccess) return e;
  return launch_persistent(product16_few_kernel<F>, max_tiles < num_sms ? max_tiles : num_sms,
                           F::SPLIT, FEW_THREADS, kFewSmem, stream, tmA, tmB, args);
}

// ---------------------------------------------------------------------------------------
// CTA pairs: 256 columns of C (the MMA's M: weight rows, 128 per CTA) x up to 256 or 512 rows (its
// N: one instruction, or two on the same weights)
// ---------------------------------------------------------------------------------------
// ROWS: that a tile may have.  SPLIT: pairs, in one cluster, that share a tile's K, each cluster one
// tile.  CHUNK: blocks of K that accumulate in TMEM, and are then added up in fp32; 0: all of them.
template <bool BT_, int ROWS_, int SPLIT_ = 1, int CHUNK_ = 0>
struct Pair {
  static constexpr bool BT = BT_;  // B [E, K, N]
  static constexpr int ROWS = ROWS_;
  static constexpr int SPLIT = SPLIT_;
  static constexpr int CHUNK = CHUNK_;
  static_assert(CHUNK == 0 || (ROWS <= 256 && SPLIT == 1), "a thread's sums");
  static constexpr int HALVES = ROWS == 512 ? 2 : 1;  // of up to 256 rows
  static constexpr int BAND = 4096 / ROWS;
};
// (the operands' ring: operand_ring.h)
constexpr uint32_t PAIR_EPI = RING * UNIT;
constexpr int PAIR_THREADS = 352;  // warp 0 producer, 1 MMA thread, 2..9 epilogue, 10 plans tiles
constexpr int PLAN_WARP = 10;
constexpr uint32_t PLANNED = 4;      // tiles ahead
constexpr int64_t MOST_PAIRS = 96;   // that a plan is made for, three to a lane
constexpr uint32_t EPI_ROW = 256 + 64;      // staged row of C: 128 columns, and an offset of 16 banks
constexpr uint32_t EPI_BUF = 32 * EPI_ROW;  // 32 rows, for each of two groups of warps
constexpr uint32_t PART_ROW = 128 * 4;      // of a split tile's sums

struct PairCtl {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tfull[2];  // of TMEM's halves
  uint64_t tempty[2];
  uint64_t mma_done;
  uint64_t planned[PLANNED];  // a tile is in the slot
  uint64_t taken[PLANNED];    // all have read it
  int4 plan[PLANNED];         // expert, first row, first column, end of the group; no expert: no more
  uint32_t tmem_base;
  int abort;
  long long total_tiles;
  GroupList list;
};
constexpr uint32_t kPairSmem = PAIR_EPI + 2 * EPI_BUF + sizeof(PairCtl) + 1024;  // + alignment slack

// Rows of half h of a tile as the MMA counts them: a multiple of 16, or 0.
template <class P>
__device__ __forceinline__ int half_height(const TileCoord& tc, int h) {
  constexpr int kMost = P::ROWS < 256 ? P::ROWS : 256;
  const int64_t left = tc.m_end - tc.m0 - 256 * h;
  return left >= kMost ? kMost : left <= 0 ? 0 : ((int)left + 15) / 16 * 16;
}

// Whether `ok` holds in all 128 threads of a group of the epilogue's warps, the same answer in each.
__device__ __forceinline__ bool all_of_group(uint32_t group, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "r"(1 + group)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ void group_sync(uint32_t group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

template <class P>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
product16_pair_kernel(const __grid_constant__ CUtensorMap tmA,    // 128 rows of A
                      const __grid_constant__ CUtensorMap tmA64,  // 64 and 32
                      const __grid_constant__ CUtensorMap tmA32,
                      const __grid_constant__ CUtensorMap tmB, const Product16Args args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  PairCtl* ctl = reinterpret_cast<PairCtl*>(smem + PAIR_EPI + 2 * EPI_BUF);
  volatile int* abort = &ctl->abort;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const int KB = (args.K + BK - 1) / BK;
  // of the CTA in its pair, its pair's leader in the cluster, and the pair's share of the tile's K
  const uint32_t cta = cluster_ctarank();
  const uint32_t rank = cta % 2, leader = cta - rank, part = cta / 2;
  const uint16_t both = (uint16_t)(0x3 << leader);
  const int kb0 = (int)((int64_t)KB * part / P::SPLIT);
  const int kb1 = (int)((int64_t)KB * (part + 1) / P::SPLIT);
  const int64_t tile0 = blockIdx.x / (2 * P::SPLIT);
  const int64_t tile_stride = gridDim.x / (2 * P::SPLIT);

  const uint32_t base = smem_u32(smem);
  auto full_bar = [&](int s) { return smem_u32(&ctl->full[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&ctl->empty[s]); };
  auto tfull_bar = [&](int s) { return smem_u32(&ctl->tfull[s]); };
  auto tempty_bar = [&](int s) { return smem_u32(&ctl->tempty[s]); };
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmA64);
    tma_prefetch_desc(&tmA32);
    tma_prefetch_desc(&tmB);
    for (uint32_t s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full_bar(s), 1);   // the leader's producer (+ both CTAs' bytes)
      mbar_init(empty_bar(s), 1);  // one commit
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull_bar(s), 1);    // one commit
      mbar_init(tempty_bar(s), 16);  // every epilogue warp of the pair
    }
    mbar_init(smem_u32(&ctl->mma_done), 1);
    for (uint32_t s = 0; s < PLANNED; ++s) {
      mbar_init(smem_u32(&ctl->planned[s]), 1);
      mbar_init(smem_u32(&ctl->taken[s]), 9 + (rank == 0));  // producer, epilogue, and MMA thread
    }
    ctl->abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish<2>();
    launch_dependents();
  }
  wait_for_previous();
  if (warp == 2) {
    int64_t row_tiles;
    const int status = list_groups<P::ROWS>(args, ctl->list, row_tiles);
    if (lane == 0) {
      ctl->total_tiles = status ? 0 : row_tiles * ((args.N + 255) / 256);
      if (status && blockIdx.x == 0) atomicCAS(args.err, 0, status);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers before any use
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const int64_t total_tiles = ctl->total_tiles;  // both CTAs of a pair agree

  // The first tile is the pair's number in the order, the others are planned: false if there is none.
  TileCoord tc;
  uint32_t slot = 0, slot_phase = 0;
  auto first_tile = [&]() {
    GroupWalk<P::ROWS, 256, P::BAND> walk;
    return tile0 < total_tiles && walk.locate(args, ctl->list, tile0, tc);
  };
  auto wait_planned = [&]() {
    return mbar_wait_sleep(smem_u32(&ctl->planned[slot]), slot_phase, abort);
  };
  auto read_planned = [&]() {  // by a thread, or a warp
    const int4 p = ctl->plan[slot];
    tc.be = p.x;
    tc.m0 = p.y;
    tc.n0 = p.z;
    tc.m_end = p.w;
    return p.x >= 0;
  };
  auto take_planned = [&]() {  // by one thread, after it (and its warp) has read
    mbar_arrive(smem_u32(&ctl->taken[slot]));
    if (++slot == PLANNED) { slot = 0; slot_phase ^= 1; }
  };
  // of one thread
  auto next_tile = [&](bool& ok) {
    if (P::SPLIT > 1 || total_tiles <= tile_stride) return false;
    ok = wait_planned();
    if (!ok) return false;
    const bool some = read_planned();
    take_planned();
    return some;
  };
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------- TMA producer -------------------------------
      // Bands of row tiles keep their rows of A in L2 while B goes by.
      const uint64_t pol_a = l2_policy_evict_last(), pol_b = l2_policy_evict_normal();
      RingPlace ring;
      RingFill fill;
      bool ok = true;
      auto free_oldest = [&](bool timed) {
        if (timed ? !mbar_wait_timed(empty_bar(fill.oldest), fill.oldest_phase)
                  : !mbar_wait_sleep(empty_bar(fill.oldest), fill.oldest_phase, abort))
          return false;
        fill.drop_oldest();
        return true;
      };
      for (bool have = first_tile(); ok && have; have = ok && next_tile(ok)) {
        const int32_t col = tc.n0 + 128 * (int)rank;
        // of each half: this CTA's first row, and its units of rows
        int32_t row[P::HALVES];
        uint32_t part[P::HALVES], units = W_UNITS;
#pragma unroll
        for (int h = 0; h < P::HALVES; ++h) {
          const int height = half_height<P>(tc, h);
          row[h] = (int32_t)tc.m0 + 256 * h + height / 2 * (int)rank;
          part[h] = half_units(height);
          units += part[h];
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          uint32_t skipped;
          const uint32_t at = ring.take(units, skipped);
          while (ok && !fill.fits(units + skipped)) ok = free_oldest(false);
          if (!ok) {
            give_up(args.err, abort);
            break;
          }
          fill.put(units + skipped);
          const uint32_t w = base + at * UNIT;
          // both CTAs' bytes are counted on the leader's barrier
          const uint32_t bar = mapa_shared(full_bar(ring.slot), leader);
          if (rank == 0) mbar_arrive_expect_tx(full_bar(ring.slot), 2 * units * UNIT);
          if constexpr (P::BT) {
            tma_load_3d_pair_hint(w, &tmB, col, kb * BK, tc.be, bar, pol_b);
            tma_load_3d_pair_hint(w + W_UNITS / 2 * UNIT, &tmB, col + 64, kb * BK, tc.be, bar,
                                  pol_b);
          } else {
            tma_load_3d_pair_hint(w, &tmB, kb * BK, col, tc.be, bar, pol_b);
          }
          uint32_t a = w + W_UNITS * UNIT;
#pragma unroll
          for (int h = 0; h < P::HALVES; ++h) {
            if (part[h] == 4) tma_load_2d_pair_hint(a, &tmA, kb * BK, row[h], bar, pol_a);
            else if (part[h] == 2) tma_load_2d_pair_hint(a, &tmA64, kb * BK, row[h], bar, pol_a);
            else if (part[h] == 1) tma_load_2d_pair_hint(a, &tmA32, kb * BK, row[h], bar, pol_a);
            a += part[h] * UNIT;
          }
          ring.next();
        }
      }
      if (!ok) give_up(args.err, abort);
      // This CTA's last loads land, and the MMAs that read them end, before it can exit (after
      // an abort the first wait runs out, which is time enough for the loads).
      while (fill.stages > 0 && free_oldest(true)) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // -------------------------------- MMA thread --------------------------------
      const uint32_t idesc0 = idesc_f16_f32(256, 0) | (P::BT ? IDESC_A_MN : 0u) |
                              (args.bf16 ? IDESC_BF16 : 0u);
      const uint64_t wdesc0 =
          P::BT ? mnmajor_sw128_desc(base, W_UNITS / 2 * UNIT) : kmajor_sw128_desc(base);
      const uint64_t adesc0 = kmajor_sw128_desc(base + W_UNITS * UNIT);
      // 16 K: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major box
      constexpr uint64_t kStepW = (P::BT ? 2048 : 32) >> 4, kStepA = 32 >> 4;
      RingPlace ring;
      uint32_t acc = 0, acc_phase = 0;  // TMEM's half that the tile's first half takes
      bool ok = true;
      for (bool have = first_tile(); ok && have; have = ok && next_tile(ok)) {
        const uint32_t n0 = half_height<P>(tc, 0), n1 = P::HALVES == 2 ? half_height<P>(tc, 1) : 0;
        const uint32_t units0 = half_units(n0), units = W_UNITS + units0 + half_units(n1);
        uint32_t d0 = tmem_base + acc * 256;
        const uint32_t d1 = tmem_base + (acc ^ 1) * 256;
        ok = mbar_wait_sleep(tempty_bar(acc), acc_phase ^ 1, abort);
        if (n1 && ok)  // (a second half that wraps around to TMEM's first is a turn later)
          ok = mbar_wait_sleep(tempty_bar(acc ^ 1), acc ? acc_phase : acc_phase ^ 1, abort);
        uint32_t more = 0;  // whether what is in TMEM is added to
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          if constexpr (P::CHUNK > 0) {
            if (kb > kb0 && (kb - kb0) % P::CHUNK == 0) {  // on to the other half
              umma_commit_pair(tfull_bar(acc), both);
              if (++acc == 2) { acc = 0; acc_phase ^= 1; }
              ok = mbar_wait_sleep(tempty_bar(acc), acc_phase ^ 1, abort);
              if (!ok) break;
              d0 = tmem_base + acc * 256;
              more = 0;
            }
          }
          ok = mbar_wait_sleep(full_bar(ring.slot), ring.phase, abort);
          if (!ok) break;
          tc_fence_after();
          uint32_t skipped;
          const uint64_t go = (uint64_t)(ring.take(units, skipped) * UNIT) >> 4;
          const uint64_t wdesc = wdesc0 + go, adesc = adesc0 + go;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_f16<2>(d0, wdesc + k * kStepW, adesc + k * kStepA, idesc0 | (n0 >> 3) << 17,
                        more || k > 0);
          if (n1) {
            const uint64_t adesc1 = adesc + ((units0 * UNIT) >> 4);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              umma_f16<2>(d1, wdesc + k * kStepW, adesc1 + k * kStepA, idesc0 | (n1 >> 3) << 17,
                          more || k > 0);
          }
          more = 1;
          umma_commit_pair(empty_bar(ring.slot), both);
          ring.next();
        }
        if (!ok) {
          give_up(args.err, abort);
          break;
        }
        for (uint32_t h = 0; h < (n1 ? 2u : 1u); ++h) {
          umma_commit_pair(tfull_bar(acc), both);
          if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
      }
      if (!ok) give_up(args.err, abort);
      // every MMA has finished before TMEM is released
      umma_commit_pair(smem_u32(&ctl->mma_done), (uint16_t)(1 << leader));
      if (!mbar_wait_timed(smem_u32(&ctl->mma_done), 0)) give_up(args.err, abort);
    }
    __syncwarp();
  } else if (warp == PLAN_WARP) {
    // ----------------------------------- plan ------------------------------------
    // Every pair follows the same plan, each for itself: the tiles in their order, each to the pair
    // that is done first by what tiles cost.  (One of every `stride` to each, as many pairs got more
    // of the full ones: 7 groups of 585 rows, 4096 x 7168, 190 us, so 170-181.)  In 82 clocks per unit
    // of 4 KB of operands, or 2 per row of MMAs.
    if (P::SPLIT == 1 && total_tiles > tile_stride) {
      const uint32_t mine = (uint32_t)tile0, pairs = (uint32_t)tile_stride;
      const uint32_t kb = (uint32_t)KB;
      auto cost_of = [&](int height) {
        const int n0 = height < 256 ? height : 256, n1 = height - n0;
        const uint32_t loads = 82 * (W_UNITS + half_units(n0) + half_units(n1)), mma = 2 * height;
        const uint32_t c = ((loads > mma ? loads : mma) * kb + 4000) >> 8;
        return c << 7;
      };
      const uint32_t full = cost_of(P::ROWS);
      // the pairs' loads above their numbers, those of pairs lane, lane + 32 and lane + 64
      uint32_t load[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) load[i] = lane + 32 * i < pairs ? lane + 32 * i : UINT32_MAX;
      const int nt = (args.N + 255) / 256;
      const bool listed = ctl->list.count >= 0;
      const int groups = listed ? ctl->list.count : args.E;
      int64_t t = 0;
      bool ok = true;
      auto push = [&](int be, int m0, int n0, int m_end) {
        ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&ctl->taken[slot]), slot_phase ^ 1, abort));
        if (!ok) return;
        if (lane == 0) {
          ctl->plan[slot] = make_int4(be, m0, n0, m_end);
          mbar_arrive(smem_u32(&ctl->planned[slot]));
        }
        if (++slot == PLANNED) { slot = 0; slot_phase ^= 1; }
      };
      // A plan of one tile for every pair takes some 8 us; where tiles are done sooner, one of every
      // `stride` (60 groups, 2155 rows, 264 x 696: planned 29.6 us, so 15.3).
      constexpr uint32_t kPlannedBlocks = 32;
      if (kb < kPlannedBlocks) {
        GroupWalk<P::ROWS, 256, P::BAND> walk;
        Turns turn(tile0, tile_stride);
        turn.next();
        for (; ok && turn.at < total_tiles && walk.locate(args, ctl->list, turn.at, tc); turn.next())
          push(tc.be, (int)tc.m0, tc.n0, (int)tc.m_end);
      }
      for (int g = 0; kb >= kPlannedBlocks && ok && g < groups; ++g) {
        int r0, r1, be;
        if (listed) {
          r0 = ctl->list.at[g].x;
          be = ctl->list.at[g].y;
          r1 = ctl->list.at[g + 1].x;
        } else {
          r0 = args.offsets[g];
          r1 = args.offsets[g + 1];
          be = args.expert_ids ? args.expert_ids[g] : g;
        }
        const int tall = (int)(((int64_t)r1 - r0) / P::ROWS), rest = r1 - r0 - tall * P::ROWS;
        const int row_tiles = tall + (rest > 0);
        const uint32_t last = rest > 0 ? cost_of((rest + 15) / 16 * 16) : full;
        for (int band = 0; ok && band < row_tiles; band += P::BAND) {
          const int end = row_tiles - band < P::BAND ? row_tiles : band + P::BAND;
          for (int col = 0; ok && col < nt; ++col) {
            for (int row = band; ok && row < end; ++row, ++t) {
              const uint32_t a = load[0] < load[1] ? load[0] : load[1];
              const uint32_t best = __reduce_min_sync(0xffffffffu, a < load[2] ? a : load[2]);
              const uint32_t pair = best & 127, cost = row == row_tiles - 1 ? last : full;
#pragma unroll
              for (int i = 0; i < 3; ++i)
                if (load[i] == best) load[i] += cost;
              if (best >= (1u << 30)) {  // the least of all: taken off everywhere
#pragma unroll
                for (int i = 0; i < 3; ++i)
                  if (load[i] != UINT32_MAX) load[i] -= best & ~127u;
              }
              // (the first of each pair it knows)
              if (pair == mine && t >= (int64_t)pairs) push(be, r0 + row * P::ROWS, col * 256, r1);
            }
          }
        }
      }
      if (ok) push(-1, 0, 0, 0);
      if (!ok && lane == 0) give_up(args.err, abort);
    }
    __syncwarp();
  } else {
    // --------------------------------- epilogue ---------------------------------
    // A lane holds a column of C.  Two groups of four warps (a warp of each TMEM quarter) take 32
    // rows in turn: through shared memory, where pairs of lanes put two columns of a row into a
    // word, and out as 256 bytes of each row.
    const uint32_t quarter = warp & 3, group = (warp - 2) >> 2;
    uint16_t* Cmat = static_cast<uint16_t*>(args.C);
    const uint64_t pol_c = l2_policy_evict_first();
    const uint32_t tempty_0 = mapa_shared(tempty_bar(0), leader);
    const uint32_t tempty_1 = mapa_shared(tempty_bar(1), leader);
    uint8_t* const staged = smem + PAIR_EPI + group * EPI_BUF;
    uint32_t acc = 0, acc_phase = 0;
    const bool odd = lane & 1;
    // (the warps of a group have barriers between them: all go on to a tile, or none)
    auto next_of_group = [&]() {
      if (P::SPLIT > 1 || total_tiles <= tile_stride) return false;
      if (!all_of_group(group, wait_planned())) {
        give_up(args.err, abort);
        return false;
      }
      const bool some = read_planned();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->taken[slot]));
      if (++slot == PLANNED) { slot = 0; slot_phase ^= 1; }
      return some;
    };
    for (bool have = first_tile(); have; have = next_of_group()) {
      const int n = tc.n0 + 128 * (int)rank + 8 * (int)(lane & 15);  // of what the lane stores
      bool ok = true;
      for (int h = 0; ok && h < P::HALVES; ++h) {
        const int height = half_height<P>(tc, h);
        if (height == 0) break;
        // the group's warps have barriers between them: all leave, or none
        ok = all_of_group(group, mbar_wait_sleep(tfull_bar(acc), acc_phase, abort));
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((quarter * 32) << 16) + acc * 256;
        auto release = [&]() {  // this warp has read its part: the MMA thread may have the half
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc ? tempty_1 : tempty_0);
        };
        auto store = [&](int c, const uint32_t (&p)[32]) {  // rows c.. of the half
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float lo = __uint_as_float(p[j]), hi = __uint_as_float(p[j + 1]);
            const uint32_t own = args.bf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
            // even lanes: row j of columns n, n + 1; odd lanes: row j + 1 of columns n - 1, n
            const uint32_t v =
                odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
            *reinterpret_cast<uint32_t*>(staged + (j + odd) * EPI_ROW +
                                         (quarter * 32 + (lane & ~1u)) * 2) = v;
          }
          group_sync(group);
          const int row0 = quarter * 8 + (int)(lane >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = row0 + 2 * i;
            const int64_t row = tc.m0 + 256 * h + c + r;
            const uint4 v = *reinterpret_cast<const uint4*>(staged + r * EPI_ROW + 16 * (lane & 15));
            if (row < tc.m_end && n < args.N)
              st_global_v4_hint(Cmat + row * (int64_t)args.N + n, v.x, v.y, v.z, v.w, pol_c);
          }
          group_sync(group);  // read before it is written again
        };
        if constexpr (P::CHUNK > 0) {
          // (the first chunk has been waited for, and the last one's turn is taken below)
          constexpr int PIECES = P::ROWS / 64;
          float sum[PIECES][32] = {};
          for (int kb = kb0;;) {
            const uint32_t from = tmem_base + ((quarter * 32) << 16) + acc * 256;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
              const int c = 32 * (int)group + 64 * i;
              if (c >= height) break;
#pragma unroll
              for (int j0 = 0; j0 < 32; j0 += 16) {
                uint32_t p[16];
                tmem_ld_32x32b_x16(from + c + j0, p);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[i][j0 + j] += __uint_as_float(p[j]);
              }
            }
            release();
            kb += P::CHUNK;
            if (kb >= kb1) break;
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            ok = all_of_group(group, mbar_wait_sleep(tfull_bar(acc), acc_phase, abort));
            if (!ok) break;
            tc_fence_after();
          }
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < PIECES; ++i) {
            const int c = 32 * (int)group + 64 * i;
            if (c >= height) break;
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) p[j] = __float_as_uint(sum[i][j]);
            store(c, p);
          }
        } else {
          if (32 * (int)group >= height) release();
          for (int c = 32 * (int)group; c < height; c += 64) {
            uint32_t p[32];
            tmem_ld_32x32b_x32(taddr + c, p);  // (past the height: whatever is there, not stored)
            tmem_ld_wait();
            if (c + 64 >= height) release();
            if constexpr (P::SPLIT > 1) {  // the part, rows of 128 columns, in the ring: it is done with
#pragma unroll
              for (int j = 0; j < 32; ++j)
                *reinterpret_cast<uint32_t*>(smem + (c + j) * PART_ROW + (quarter * 32 + lane) * 4) = p[j];
            } else {
              store(c, p);
            }
          }
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok) {
        give_up(args.err, abort);
        break;
      }
    }
  }

  if constexpr (P::SPLIT > 1) {
    // Each pair adds up some of the tile's rows, in the pairs' order.  (A pair that gave up has said
    // so, and the sums mean nothing.)  The cluster's barrier below is the one before any CTA goes.
    static_assert(P::ROWS * PART_ROW <= RING * UNIT && P::HALVES == 1, "part");
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && warp < PLAN_WARP && tile0 < total_tiles) {
      GroupWalk<P::ROWS, 256, P::BAND> again;
      again.locate(args, ctl->list, tile0, tc);
      const int height = half_height<P>(tc, 0);
      const int n = tc.n0 + 128 * (int)rank + 8 * (int)(lane & 15);
      const int first = (int)part + P::SPLIT * (int)((threadIdx.x - 64) / 16);
      for (int r = first; r < height; r += P::SPLIT * 16) {
        const int64_t row = tc.m0 + r;
        if (row >= tc.m_end || n >= args.N) continue;  // N is a multiple of 8
        float4 v[2][P::SPLIT];
#pragma unroll
        for (int s = 0; s < P::SPLIT; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[h][s] = load_cluster_f4(
                mapa_shared(base + r * PART_ROW + 32 * (lane & 15) + 16 * h, 2 * s + rank));
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int s = 1; s < P::SPLIT; ++s) {
            v[h][0].x += v[h][s].x;
            v[h][0].y += v[h][s].y;
            v[h][0].z += v[h][s].z;
            v[h][0].w += v[h][s].w;
          }
          const float4 x = v[h][0];
          w[2 * h] = args.bf16 ? pack_bf16x2(x.x, x.y) : pack_f16x2(x.x, x.y);
          w[2 * h + 1] = args.bf16 ? pack_bf16x2(x.z, x.w) : pack_f16x2(x.z, x.w);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.C) + row * (int64_t)args.N + n) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // the pair's MMAs and remote arrivals are finished before either CTA frees TMEM or exits
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, 512);
  }
}

template <class P>
cudaError_t launch_pair(const Product16Args& args, int num_sms, cudaStream_t stream) {
  static_assert(kPairSmem <= 227 * 1024, "shared memory per CTA");
  CUtensorMap tmA, tmA64, tmA32, tmB;
  const uint64_t a_dims[2] = {(uint64_t)args.K, (uint64_t)args.M_total};
  const uint64_t b_dims[3] = {(uint64_t)(P::BT ? args.N : args.K),
                              (uint64_t)(P::BT ? args.K : args.N), (uint64_t)args.num_experts};
  if (!encode_swizzled(&tmA, 2, args.A, 2, a_dims, 128) ||
      !encode_swizzled(&tmA64, 2, args.A, 2, a_dims, 64) ||
      !encode_swizzled(&tmA32, 2, args.A, 2, a_dims, 32) ||
      !encode_swizzled(&tmB, 2, args.B, 3, b_dims, P::BT ? BK : 128))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<product16_pair_kernel<P>>(kPairSmem);
  if (e != cudaSuccess) return e;
  int64_t units = num_sms / (2 * P::SPLIT);
  if (units > MOST_PAIRS) units = MOST_PAIRS;
  const int64_t tiles = most_tiles(args, P::ROWS, 256);
  return launch_persistent(product16_pair_kernel<P>, tiles < units ? tiles : units, 2 * P::SPLIT,
                           PAIR_THREADS, kPairSmem, stream, tmA, tmA64, tmA32, tmB, args);
}

template <class F>
int64_t few_at_once() {
  return clusters_at_once<product16_few_kernel<F>>(F::SPLIT, FEW_THREADS, kFewSmem);
}
template <class P>
int64_t pairs_at_once() {
  return clusters_at_once<product16_pair_kernel<P>>(2 * P::SPLIT, PAIR_THREADS, kPairSmem);
}

// How many clusters the device holds at once of a form whose K is shared `split` ways: those given (of
// 2, 4 and 8 CTAs), or the current device's.
template <bool BT>
struct AtOnce {
  const int32_t* given;
  int64_t few(int split) const {
    if (given) return given[split == 2 ? 0 : split == 4 ? 1 : 2];
    return split == 2   ? few_at_once<Few<BT, 2>>()
           : split == 4 ? few_at_once<Few<BT, 4>>()
                        : few_at_once<Few<BT, 8>>();
  }
  int64_t pairs(int split) const {
    if (given) return given[split == 2 ? 1 : 2];
    return split == 2 ? pairs_at_once<Pair<BT, 128, 2>>() : pairs_at_once<Pair<BT, 128, 4>>();
  }
};

template <bool BT>
Product16Plan choose(const Product16Args& a, int num_sms, const AtOnce<BT>& at_once) {
  const auto few = [](int split) { return Product16Plan{FEW_ROWS, FEW_COLS, 1, split, 0}; };
  const auto pair = [](int rows, int split, int chunk) {
    return Product16Plan{rows, 256, 2, split, chunk};
  };
  // A tile's K is shared where that leaves each of the tile's CTAs a part and an SM (a second round of
  // clusters costs more than sharing gains: 1000 rows, 512 x 2048, shared by four pairs 20.7 us, by two
  // 12.8).
  const int64_t few_tiles = most_tiles(a, FEW_ROWS, FEW_COLS);
  const int64_t blocks = (a.K + BK - 1) / BK;
  // whether one accumulator will do for each of `split` parts of K
  const int most_blocks = a.bf16 ? MOST_BLOCKS_BF16 : MOST_BLOCKS_FP16;
  auto one_sum = [&](int split) { return (blocks + split - 1) / split <= most_blocks; };
  if (blocks >= 16 && one_sum(8) && few_tiles <= at_once.few(8)) return few(8);
  if (blocks >= 8 && one_sum(4) && few_tiles <= at_once.few(4)) return few(4);
  if (blocks >= 4 && one_sum(2) && few_tiles <= at_once.few(2)) return few(2);
  // Up to 8 rows per group on average, most groups are one tile of 32 rows: less to load and to
  // set up than in tiles of pairs (64 groups of 1 row, 2048 x 2048: 81 us against 88; 16 of 8, 2048
  // x 4096: 45 and 48).  With more of them a few groups can hold many, and each reads its weights
  // once per 32 rows (4027 rows over 128 groups, the largest 753, 4096 x 2048: 422 us against 330;
  // 4096 rows in one of them 222 and 51; 16 rows in each 327 and 322).
  if (one_sum(1) && (a.M_total <= FEW_ROWS || a.M_total <= (int64_t)8 * a.E))
    return few(1);
  const int64_t units = num_sms / 2;
  // about how many tiles there are: the last of a group is half full
  auto tiles = [&](int rows) {
    const int64_t row_tiles =
        a.E == 1 ? (a.M_total + rows - 1) / rows : a.M_total / rows + (a.E + 1) / 2;
    return (row_tiles > a.E ? row_tiles : a.E) * ((a.N + 255) / 256);
  };
  // What takes least of tiles of 512, 256, 128 or 64 rows, or of 128 whose K two or four pairs share: a
  // tile so many units of 4 KB per block of 64 K, and about 48 units to start and end it; of more tiles
  // than pairs the last ones leave some pairs idle, for half a tile or, of 512 rows, one.  Where little
  // is between them the higher ones: groups of many rows read their weights less often.  With each
  // height, us: 64 groups of 260 rows, 7168 x 2048: 496 in tiles of 256 and 400 of 512; 7 of 585, 4096 x
  // 7168: 235 of 128, 170-181 of 256, 220 of 512; 8177 rows over 128 groups, the largest 1517, 4096 x 2048:
  // 367 of 128, 345 of 256; 545 rows, 3000 x 1256: 18.9 of 64, 13.3 of 128, 14.7 of 256; 128 rows, 4096
  // x 4096: 21.4, shared by two pairs 16.8; 1000 rows, 512 x 2048: 13.6, by two 12.8.
  auto cost = [&](int rows, int split) {
    const int64_t n = tiles(rows);
    const double height = (double)a.M_total * ((a.N + 255) / 256) / n;
    const double kb = (double)((blocks + split - 1) / split), ends = split == 1 ? 48 : split == 2 ? 96 : 128;
    const double one = kb * (4 + height / 64) + ends;
    if (n * split <= units) return one;
    return one * n * split / units + (rows == 512 ? 1.2 : 0.6) * (kb * (4 + rows / 64) + ends);
  };
  const double c64 = 1.06 * cost(64, 1), c128 = 1.03 * cost(128, 1), c256 = cost(256, 1);
  const double c512 = cost(512, 1);
  const double low = c64 < c128 ? c64 : c128, high = c256 <= c512 ? c256 : c512;
  const double least = !one_sum(1) ? c256 : low < high ? low : high;
  const int64_t most = most_tiles(a, 128, 256);
  if (blocks >= 16 && one_sum(4) && cost(128, 4) < least && cost(128, 4) < cost(128, 2) &&
      most <= at_once.pairs(4))
    return pair(128, 4, 0);
  if (blocks >= 8 && one_sum(2) && cost(128, 2) < least && most <= at_once.pairs(2))
    return pair(128, 2, 0);
  if (!one_sum(1)) return pair(256, 1, CHUNK_BLOCKS * BK);
  return pair(c256 == least ? 256 : c512 == least ? 512 : c128 == least ? 128 : 64, 1, 0);
}

template <bool BT>
cudaError_t launch_chosen(const Product16Args& a, int num_sms, cudaStream_t stream) {
  const Product16Plan p = choose<BT>(a, num_sms, AtOnce<BT>{nullptr});
  if (p.ctas == 1) {
    const int64_t tiles = most_tiles(a, FEW_ROWS, FEW_COLS);
    switch (p.split) {
      case 8: return launch_few<Few<BT, 8>>(a, tiles, num_sms, stream);
      case 4: return launch_few<Few<BT, 4>>(a, tiles, num_sms, stream);
      case 2: return launch_few<Few<BT, 2>>(a, tiles, num_sms, stream);
      default: return launch_few<Few<BT, 1>>(a, tiles, num_sms, stream);
    }
  }
  if (p.chunk) return launch_pair<Pair<BT, 256, 1, CHUNK_BLOCKS>>(a, num_sms, stream);
  if (p.split == 4) return launch_pair<Pair<BT, 128, 4>>(a, num_sms, stream);
  if (p.split == 2) return launch_pair<Pair<BT, 128, 2>>(a, num_sms, stream);
  switch (p.rows) {
    case 512: return launch_pair<Pair<BT, 512>>(a, num_sms, stream);
    case 256: return launch_pair<Pair<BT, 256>>(a, num_sms, stream);
    case 128: return launch_pair<Pair<BT, 128>>(a, num_sms, stream);
    default: return launch_pair<Pair<BT, 64>>(a, num_sms, stream);
  }
}

}  // namespace g16

cudaError_t launch_product16(const Product16Args& a, int num_sms, cudaStream_t stream) {
  return a.transposed ? g16::launch_chosen<true>(a, num_sms, stream)
                      : g16::launch_chosen<false>(a, num_sms, stream);
}

Product16Plan plan_product16(const Product16Args& a, int num_sms, const int32_t* clusters) {
  return a.transposed ? g16::choose<true>(a, num_sms, g16::AtOnce<true>{clusters})
                      : g16::choose<false>(a, num_sms, g16::AtOnce<false>{clusters});
}

}  // namespace bsfp8
