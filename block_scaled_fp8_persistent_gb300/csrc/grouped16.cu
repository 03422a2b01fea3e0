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
// Roles (6 warps): warp 0 TMA producer; warp 1 TMEM owner and, in CTA 0, the MMA thread (per 64 K
// four MMAs of K = 16 and one commit); warps 2-5 epilogue, TMEM lanes 32 * (w % 4)..: rows of
// C, which are stored as 32-byte sectors while the next tile accumulates in the other half of
// TMEM.
//
// Tiles: a CTA pair takes 256 rows x 256 columns (each CTA 128 rows and half of B); one CTA 128 x
// 256 or 32 x 128.  With few rows per expert the weights' bytes bound the product, and what counts
// is how many of them are in flight: tiles of 32 rows keep 8 stages of 16 KB of weights per SM, and
// the MMA computes 128 rows of which the last 96 (whatever follows in shared memory) are not read.
#include <atomic>
#include "expert_ops.cuh"
#include "ptx.cuh"
#include "sched.cuh"

namespace bsfp8 {
namespace g16 {

constexpr int BK = 64;  // elements: 128 bytes
constexpr int THREADS = 192;

// The tiles that CTA (or pair) `unit` of `units` takes: one of every `units`, in each round the next
// place.  Row tiles of a group follow one another in the numbering, the last often a small one; at
// a fixed place some units would get all the full ones (groups of 260 rows, 64 of them, 7168 x
// 2048: 484 us, in turns 414).
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

template <int CG_, int BN_, int ROWS_, bool BT_, int STAGES_>
struct Cfg {
  static constexpr int CG = CG_;          // CTAs per tile
  static constexpr int BN = BN_;          // tile columns
  static constexpr int ROWS = ROWS_;      // rows of A per CTA
  static constexpr int BM = CG * ROWS;    // tile rows
  static constexpr bool BT = BT_;         // B [E, K, N]
  static constexpr int STAGES = STAGES_;
  static constexpr int EPI_WARPS = ROWS / 32;  // that hold rows
  static constexpr int B_ROWS = BN / CG;       // columns of C whose weights a CTA loads
  static constexpr uint32_t A_STAGE = ROWS * BK * 2;
  static constexpr uint32_t B_STAGE = B_ROWS * BK * 2;
  static constexpr uint32_t B_BOX = BT ? 64 * BK * 2 : B_STAGE;
  static constexpr uint32_t STAGE_TX = (A_STAGE + B_STAGE) * CG;
  static constexpr uint32_t SMEM_A = 0;
  static constexpr uint32_t SMEM_B = SMEM_A + STAGES * A_STAGE;
  static constexpr uint32_t SMEM_CTL = SMEM_B + STAGES * B_STAGE;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr uint32_t IDESC = idesc_f16_f32(128 * CG, BN) | (BT ? IDESC_B_MN : 0u);
  // what the MMA of the last stage reads past A ends inside B
  static_assert(ROWS == 128 || (128 - ROWS) * BK * 2 <= (int)(STAGES * B_STAGE), "A's overhang");
  // row tiles that share a column of B within a wave (as in the 8-bit kernels)
  static constexpr int TILE_BAND = CG == 2 ? 16 : 1;
};

template <class C>
struct Ctl {
  uint64_t full[C::STAGES];
  uint64_t empty[C::STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int valid;
  int pad;
  long long total_tiles;
};

template <class C>
constexpr uint32_t smem_bytes() {
  return C::SMEM_CTL + sizeof(Ctl<C>) + 1024;  // + alignment slack
}

template <class C>
__global__ void __launch_bounds__(THREADS, 1)
product16_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const Product16Args args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl<C>* ctl = reinterpret_cast<Ctl<C>*>(smem + C::SMEM_CTL);
  volatile int* abort = &ctl->abort;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const int KB = (args.K + BK - 1) / BK;
  const uint32_t rank = C::CG == 2 ? cluster_ctarank() : 0;
  const int64_t tile0 = blockIdx.x / C::CG;
  const int64_t tile_stride = gridDim.x / C::CG;

  if (warp == 0) {
    int64_t row_tiles;
    const int status = check_groups<C::BM>(args.offsets, args.expert_ids, args.E,
                                           args.num_experts, args.M_total, row_tiles);
    if (lane == 0) {
      ctl->valid = status == 0;
      ctl->total_tiles = row_tiles * ((args.N + C::BN - 1) / C::BN);
      ctl->abort = 0;
      if (status && blockIdx.x == 0) atomicCAS(args.err, 0, status);
    }
  }
  __syncthreads();
  const int64_t total_tiles = ctl->total_tiles;
  if (!ctl->valid || tile0 >= total_tiles) return;  // both CTAs of a pair agree

  const uint32_t sA = smem_u32(smem + C::SMEM_A);
  const uint32_t sB = smem_u32(smem + C::SMEM_B);
  auto full_bar = [&](int s) { return smem_u32(&ctl->full[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&ctl->empty[s]); };
  auto tfull_bar = [&](int s) { return smem_u32(&ctl->tfull[s]); };
  auto tempty_bar = [&](int s) { return smem_u32(&ctl->tempty[s]); };
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);   // the leader's producer (+ both CTAs' bytes)
      mbar_init(empty_bar(s), 1);  // one commit
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull_bar(s), 1);                       // one commit
      mbar_init(tempty_bar(s), C::EPI_WARPS * C::CG);   // every epilogue warp of the pair
    }
    mbar_init(smem_u32(&ctl->mma_done), 1);
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc<C::CG>(smem_u32(&ctl->tmem_base), C::TMEM_COLS);
    tmem_relinquish<C::CG>();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C::CG == 2) cluster_sync();  // the peer's barriers before any use
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  GroupedScheduler<C::BM, C::BN, C::TILE_BAND> sched;
  TileCoord tc;
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------- TMA producer -------------------------------
      // Pairs walk in bands whose rows of A stay in L2 while B goes by; decode-sized tiles read
      // every weight once.
      const uint64_t pol_a = l2_policy_evict_last();
      const uint64_t pol_b = C::ROWS == 32 ? l2_policy_evict_first() : l2_policy_evict_normal();
      uint32_t stage = 0, phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (Turns t(tile0, tile_stride); ok && t.at < total_tiles; t.next()) {
        if (!sched.locate(args, t.at, tc)) break;
        const int32_t a_row = (int32_t)(tc.m0 + C::ROWS * rank);
        const int32_t col = tc.n0 + C::B_ROWS * rank;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_sleep(empty_bar(stage), phase ^ 1, abort)) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          const uint32_t a = sA + stage * C::A_STAGE, b = sB + stage * C::B_STAGE;
          if constexpr (C::CG == 1) {
            mbar_arrive_expect_tx(full_bar(stage), C::STAGE_TX);
            tma_load_2d_hint(a, &tmA, kb * BK, a_row, full_bar(stage), pol_a);
            if constexpr (C::BT) {
              for (int i = 0; i < C::B_ROWS / 64; ++i)
                tma_load_3d_hint(b + i * C::B_BOX, &tmB, col + 64 * i, kb * BK, tc.be,
                                 full_bar(stage), pol_b);
            } else {
              tma_load_3d_hint(b, &tmB, kb * BK, col, tc.be, full_bar(stage), pol_b);
            }
          } else {
            // both CTAs' bytes are counted on the leader's barrier
            const uint32_t bar = mapa_shared(full_bar(stage), 0);
            if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), C::STAGE_TX);
            tma_load_2d_pair_hint(a, &tmA, kb * BK, a_row, bar, pol_a);
            if constexpr (C::BT) {
              for (int i = 0; i < C::B_ROWS / 64; ++i)
                tma_load_3d_pair_hint(b + i * C::B_BOX, &tmB, col + 64 * i, kb * BK, tc.be, bar,
                                      pol_b);
            } else {
              tma_load_3d_pair_hint(b, &tmB, kb * BK, col, tc.be, bar, pol_b);
            }
          }
          ++issued;
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
      }
      // This CTA's last loads land, and the MMAs that read them end, before it can exit (after
      // an abort the first wait runs out, which is time enough for the loads).
      const int64_t pending = issued < C::STAGES ? issued : C::STAGES;
      for (int64_t i = 0; i < pending; ++i) {
        stage = (stage + C::STAGES - 1) % C::STAGES;
        if (stage == C::STAGES - 1) phase ^= 1;
        if (!mbar_wait_timed(empty_bar(stage), phase)) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // -------------------------------- MMA thread --------------------------------
      const uint32_t idesc = C::IDESC | (args.bf16 ? IDESC_BF16 : 0u);
      const uint64_t adesc0 = kmajor_sw128_desc(sA);
      const uint64_t bdesc0 = C::BT ? mnmajor_sw128_desc(sB, C::B_BOX) : kmajor_sw128_desc(sB);
      // 16 K: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major box
      constexpr uint64_t kStepA = 32 >> 4, kStepB = (C::BT ? 2048 : 32) >> 4;
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      for (Turns t(tile0, tile_stride); ok && t.at < total_tiles; t.next()) {
        if (!sched.locate(args, t.at, tc)) break;
        if (!mbar_wait_sleep(tempty_bar(acc), acc_phase ^ 1, abort)) {
          give_up(args.err, abort);
          break;
        }
        const uint32_t d = tmem_base + acc * C::BN;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_sleep(full_bar(stage), phase, abort)) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t adesc = adesc0 + ((stage * C::A_STAGE) >> 4);
          const uint64_t bdesc = bdesc0 + ((stage * C::B_STAGE) >> 4);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_f16<C::CG>(d, adesc + k * kStepA, bdesc + k * kStepB, idesc, (kb | k) > 0);
          if constexpr (C::CG == 1) umma_commit(empty_bar(stage));
          else umma_commit_pair(empty_bar(stage), 0x3);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if constexpr (C::CG == 1) umma_commit(tfull_bar(acc));
        else umma_commit_pair(tfull_bar(acc), 0x3);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      // every MMA has finished before TMEM is released
      if constexpr (C::CG == 1) umma_commit(smem_u32(&ctl->mma_done));
      else umma_commit_pair(smem_u32(&ctl->mma_done), 0x1);
      if (!mbar_wait_timed(smem_u32(&ctl->mma_done), 0)) give_up(args.err, abort);
    }
    __syncwarp();
  } else if ((warp & 3) < C::EPI_WARPS) {
    // --------------------------------- epilogue ---------------------------------
    const uint32_t quarter = warp & 3;
    uint16_t* Cmat = static_cast<uint16_t*>(args.C);
    const bool wide = (reinterpret_cast<uintptr_t>(args.C) & 31) == 0 && args.N % 16 == 0;
    const uint64_t pol_c = l2_policy_evict_first();
    uint32_t acc = 0, acc_phase = 0;
    for (Turns t(tile0, tile_stride); t.at < total_tiles; t.next()) {
      if (!sched.locate(args, t.at, tc)) break;
      const int64_t row = tc.m0 + C::ROWS * rank + quarter * 32 + lane;
      if (!__all_sync(0xffffffffu, mbar_wait_sleep(tfull_bar(acc), acc_phase, abort))) {
        if (lane == 0) give_up(args.err, abort);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((quarter * 32) << 16) + acc * C::BN;
      uint16_t* dst = Cmat + row * (int64_t)args.N + tc.n0;
      const int cols = args.N - tc.n0;  // that are left of the matrix
#pragma unroll 1
      for (int c = 0; c < C::BN; c += 32) {
        uint32_t p[32];
        tmem_ld_32x32b_x32(taddr + c, p);
        tmem_ld_wait();
        if (c + 32 == C::BN) {  // TMEM is read: the MMA thread may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0)
            mbar_arrive_cluster_or_local<C::CG>(C::CG == 2 ? mapa_shared(tempty_bar(acc), 0)
                                                           : tempty_bar(acc));
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
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  }

  tc_fence_before();
  __syncthreads();
  // the pair's MMAs and remote arrivals are finished before either CTA frees TMEM or exits
  if constexpr (C::CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<C::CG>(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------
// CTA pairs: 256 columns of C (the MMA's M: weight rows, 128 per CTA) x up to 256 or 512 rows (its
// N: one instruction, or two on the same weights)
// ---------------------------------------------------------------------------------------
// HALVES: of 256 rows that a tile may have.
template <bool BT_, int HALVES_>
struct Pair {
  static constexpr bool BT = BT_;  // B [E, K, N]
  static constexpr int HALVES = HALVES_;
  static constexpr int ROWS = 256 * HALVES;
  static constexpr int BAND = HALVES == 2 ? 8 : 16;
};
constexpr uint32_t UNIT = 4096;              // 32 rows of 128 bytes: what a stage of the ring counts in
constexpr uint32_t RING = 51;                // units
constexpr uint32_t W_UNITS = 4;              // a CTA's 128 weight rows
constexpr uint32_t MAX_STAGES = 10;          // barriers: one more than the smallest stages that fit
constexpr uint32_t PAIR_EPI = RING * UNIT;
constexpr int PAIR_THREADS = 320;
constexpr uint32_t EPI_ROW = 256 + 64;      // staged row of C: 128 columns, and an offset of 16 banks
constexpr uint32_t EPI_BUF = 32 * EPI_ROW;  // 32 rows, for each of two groups of warps

struct PairCtl {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tfull[2];  // of TMEM's halves
  uint64_t tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int valid;
  int pad;
  long long total_tiles;
};
constexpr uint32_t kPairSmem = PAIR_EPI + 2 * EPI_BUF + sizeof(PairCtl) + 1024;  // + alignment slack

// The operands' ring.  A stage is as large as its tile needs it: the weights' units, and of each
// half's rows as many as they fill, so that short tiles have more stages in flight (51 units: four
// stages of 512 rows, six of 256, nine of 32).  Producer and MMA thread place stages by the same
// rule: one behind the other, at the start where the end is too near.
struct RingPlace {
  uint32_t head = 0, slot = 0, phase = 0;
  // start of a stage of `units`; the barriers' slot and phase are those of the members
  __device__ uint32_t take(uint32_t units, uint32_t& skipped) {
    const bool wraps = head + units > RING;
    skipped = wraps ? RING - head : 0;
    const uint32_t at = wraps ? 0 : head;
    head = at + units;
    return at;
  }
  __device__ void next() {
    if (++slot == MAX_STAGES) { slot = 0; phase ^= 1; }
  }
};

// Rows of half h of a tile as the MMA counts them: a multiple of 16, or 0.
__device__ __forceinline__ int half_height(const TileCoord& tc, int h) {
  const int64_t left = tc.m_end - tc.m0 - 256 * h;
  return left >= 256 ? 256 : left <= 0 ? 0 : ((int)left + 15) / 16 * 16;
}

// Units of half h's rows in a stage: 128, 64 or 32 rows, the box of one load (several small ones
// cost more than the rows they save: 64 groups of 160 rows 350 us with 3 of 32 rows, 313 with 128).
__device__ __forceinline__ uint32_t half_units(int height) {
  return height > 128 ? 4 : height > 64 ? 2 : height > 0 ? 1 : 0;
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
  const uint32_t rank = cluster_ctarank();
  const int64_t tile0 = blockIdx.x / 2;
  const int64_t tile_stride = gridDim.x / 2;

  if (warp == 0) {
    int64_t row_tiles;
    const int status = check_groups<P::ROWS>(args.offsets, args.expert_ids, args.E,
                                             args.num_experts, args.M_total, row_tiles);
    if (lane == 0) {
      ctl->valid = status == 0;
      ctl->total_tiles = row_tiles * ((args.N + 255) / 256);
      ctl->abort = 0;
      if (status && blockIdx.x == 0) atomicCAS(args.err, 0, status);
    }
  }
  __syncthreads();
  const int64_t total_tiles = ctl->total_tiles;
  if (!ctl->valid || tile0 >= total_tiles) return;  // both CTAs of a pair agree

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
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers before any use
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  GroupedScheduler<P::ROWS, 256, P::BAND> sched;
  TileCoord tc;
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------- TMA producer -------------------------------
      // Bands of row tiles keep their rows of A in L2 while B goes by.
      const uint64_t pol_a = l2_policy_evict_last(), pol_b = l2_policy_evict_normal();
      RingPlace ring;
      uint32_t oldest = 0, oldest_phase = 0;      // the barrier of the oldest stage in the ring
      uint32_t stages = 0, used = 0;              // in the ring: stages, units (and skipped ones)
      uint64_t sizes = 0;                         // of the stages in the ring, the oldest's first
      constexpr int kBits = 6;
      bool ok = true;
      auto free_oldest = [&](bool timed) {
        if (timed ? !mbar_wait_timed(empty_bar(oldest), oldest_phase)
                  : !mbar_wait_sleep(empty_bar(oldest), oldest_phase, abort))
          return false;
        if (++oldest == MAX_STAGES) { oldest = 0; oldest_phase ^= 1; }
        used -= (uint32_t)(sizes & ((1u << kBits) - 1));
        sizes >>= kBits;
        --stages;
        return true;
      };
      for (Turns t(tile0, tile_stride); ok && t.at < total_tiles; t.next()) {
        if (!sched.locate(args, t.at, tc)) break;
        const int32_t col = tc.n0 + 128 * (int)rank;
        // of each half: this CTA's first row, and its units of rows
        int32_t row[P::HALVES];
        uint32_t part[P::HALVES], units = W_UNITS;
#pragma unroll
        for (int h = 0; h < P::HALVES; ++h) {
          const int height = half_height(tc, h);
          row[h] = (int32_t)tc.m0 + 256 * h + height / 2 * (int)rank;
          part[h] = half_units(height);
          units += part[h];
        }
        for (int kb = 0; kb < KB; ++kb) {
          uint32_t skipped;
          const uint32_t at = ring.take(units, skipped);
          while (ok && (used + units + skipped > RING || stages + 1 == MAX_STAGES))
            ok = free_oldest(false);
          if (!ok) {
            give_up(args.err, abort);
            break;
          }
          used += units + skipped;
          sizes |= (uint64_t)(units + skipped) << (kBits * stages);
          ++stages;
          const uint32_t w = base + at * UNIT;
          // both CTAs' bytes are counted on the leader's barrier
          const uint32_t bar = mapa_shared(full_bar(ring.slot), 0);
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
      // This CTA's last loads land, and the MMAs that read them end, before it can exit (after
      // an abort the first wait runs out, which is time enough for the loads).
      while (stages > 0 && free_oldest(true)) {
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
      for (Turns t(tile0, tile_stride); ok && t.at < total_tiles; t.next()) {
        if (!sched.locate(args, t.at, tc)) break;
        const uint32_t n0 = half_height(tc, 0), n1 = P::HALVES == 2 ? half_height(tc, 1) : 0;
        const uint32_t units0 = half_units(n0), units = W_UNITS + units0 + half_units(n1);
        const uint32_t d0 = tmem_base + acc * 256, d1 = tmem_base + (acc ^ 1) * 256;
        ok = mbar_wait_sleep(tempty_bar(acc), acc_phase ^ 1, abort);
        if (n1 && ok)  // (a second half that wraps around to TMEM's first is a turn later)
          ok = mbar_wait_sleep(tempty_bar(acc ^ 1), acc ? acc_phase : acc_phase ^ 1, abort);
        for (int kb = 0; ok && kb < KB; ++kb) {
          ok = mbar_wait_sleep(full_bar(ring.slot), ring.phase, abort);
          if (!ok) break;
          tc_fence_after();
          uint32_t skipped;
          const uint64_t go = (uint64_t)(ring.take(units, skipped) * UNIT) >> 4;
          const uint64_t wdesc = wdesc0 + go, adesc = adesc0 + go;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_f16<2>(d0, wdesc + k * kStepW, adesc + k * kStepA, idesc0 | (n0 >> 3) << 17,
                        (kb | k) > 0);
          if (n1) {
            const uint64_t adesc1 = adesc + ((units0 * UNIT) >> 4);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              umma_f16<2>(d1, wdesc + k * kStepW, adesc1 + k * kStepA, idesc0 | (n1 >> 3) << 17,
                          (kb | k) > 0);
          }
          umma_commit_pair(empty_bar(ring.slot), 0x3);
          ring.next();
        }
        if (!ok) {
          give_up(args.err, abort);
          break;
        }
        for (uint32_t h = 0; h < (n1 ? 2u : 1u); ++h) {
          umma_commit_pair(tfull_bar(acc), 0x3);
          if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
      }
      // every MMA has finished before TMEM is released
      umma_commit_pair(smem_u32(&ctl->mma_done), 0x1);
      if (!mbar_wait_timed(smem_u32(&ctl->mma_done), 0)) give_up(args.err, abort);
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
    const uint32_t tempty_0 = mapa_shared(tempty_bar(0), 0), tempty_1 = mapa_shared(tempty_bar(1), 0);
    uint8_t* const staged = smem + PAIR_EPI + group * EPI_BUF;
    uint32_t acc = 0, acc_phase = 0;
    const bool odd = lane & 1;
    for (Turns t(tile0, tile_stride); t.at < total_tiles; t.next()) {
      if (!sched.locate(args, t.at, tc)) break;
      const int n = tc.n0 + 128 * (int)rank + 8 * (int)(lane & 15);  // of what the lane stores
      bool ok = true;
      for (int h = 0; ok && h < P::HALVES; ++h) {
        const int height = half_height(tc, h);
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
        if (32 * (int)group >= height) release();
        for (int c = 32 * (int)group; c < height; c += 64) {
          uint32_t p[32];
          tmem_ld_32x32b_x32(taddr + c, p);  // (past the height: whatever is there, not stored)
          tmem_ld_wait();
          if (c + 64 >= height) release();
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
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok) {
        give_up(args.err, abort);
        break;
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
  if (!encode_swizzled(&tmA, false, args.A, 2, a_dims, 128) ||
      !encode_swizzled(&tmA64, false, args.A, 2, a_dims, 64) ||
      !encode_swizzled(&tmA32, false, args.A, 2, a_dims, 32) ||
      !encode_swizzled(&tmB, false, args.B, 3, b_dims, P::BT ? BK : 128))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];  // per device; several host threads may launch
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(product16_pair_kernel<P>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)kPairSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  // more tiles than this there are not (the offsets live on the device)
  const int64_t max_tiles = ((args.M_total + P::ROWS - 1) / P::ROWS + args.E) * ((args.N + 255) / 256);
  const int64_t units = num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((max_tiles < units ? max_tiles : units) * 2));
  cfg.blockDim = dim3(PAIR_THREADS);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, product16_pair_kernel<P>, tmA, tmA64, tmA32, tmB, args);
}

template <class C>
cudaError_t launch(const Product16Args& args, int num_sms, cudaStream_t stream) {
  static_assert(smem_bytes<C>() <= 227 * 1024, "shared memory per CTA");
  CUtensorMap tmA, tmB;
  const uint64_t a_dims[2] = {(uint64_t)args.K, (uint64_t)args.M_total};
  const uint64_t inner = C::BT ? args.N : args.K, outer = C::BT ? args.K : args.N;
  const uint64_t b_dims[3] = {inner, outer, (uint64_t)args.num_experts};
  if (!encode_swizzled(&tmA, false, args.A, 2, a_dims, C::ROWS) ||
      !encode_swizzled(&tmB, false, args.B, 3, b_dims, C::BT ? BK : C::B_ROWS))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];  // per device; several host threads may launch
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(product16_kernel<C>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes<C>());
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  // more tiles than this there are not (the offsets live on the device)
  const int64_t max_row_tiles = (args.M_total + C::BM - 1) / C::BM + args.E;
  const int64_t max_tiles = max_row_tiles * ((args.N + C::BN - 1) / C::BN);
  const int64_t units = num_sms / C::CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((max_tiles < units ? max_tiles : units) * C::CG));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes<C>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, product16_kernel<C>, tmA, tmB, args);
}

template <bool BT>
cudaError_t choose(const Product16Args& a, int num_sms, cudaStream_t stream) {
  if (a.M_total <= (int64_t)32 * a.E)
    return launch<Cfg<1, 128, 32, BT, 9>>(a, num_sms, stream);
  if (a.M_total <= (int64_t)128 * a.E)
    return launch<Cfg<1, 256, 128, BT, 4>>(a, num_sms, stream);
  const int64_t tall = (a.M_total / 512 + a.E / 2) * ((a.N + 255) / 256);
  return tall >= 6 * (num_sms / 2) ? launch_pair<Pair<BT, 2>>(a, num_sms, stream)
                                   : launch_pair<Pair<BT, 1>>(a, num_sms, stream);
}

}  // namespace g16

cudaError_t launch_product16(const Product16Args& a, int num_sms, cudaStream_t stream) {
  return a.transposed ? g16::choose<true>(a, num_sms, stream)
                      : g16::choose<false>(a, num_sms, stream);
}

}  // namespace bsfp8
