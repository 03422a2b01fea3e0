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
constexpr int EPI_WARP0 = 2;

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
      for (int64_t t = tile0; ok && t < total_tiles; t += tile_stride) {
        if (!sched.locate(args, t, tc)) break;
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
      for (int64_t t = tile0; ok && t < total_tiles; t += tile_stride) {
        if (!sched.locate(args, t, tc)) break;
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
    for (int64_t t = tile0; t < total_tiles; t += tile_stride) {
      if (!sched.locate(args, t, tc)) break;
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
  return launch<Cfg<2, 256, 128, BT, 6>>(a, num_sms, stream);
}

}  // namespace g16

cudaError_t launch_product16(const Product16Args& a, int num_sms, cudaStream_t stream) {
  return a.transposed ? g16::choose<true>(a, num_sms, stream)
                      : g16::choose<false>(a, num_sms, stream);
}

}  // namespace bsfp8
