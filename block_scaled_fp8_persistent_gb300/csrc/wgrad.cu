// Weight gradients of products grouped by expert, for sm_103a (persistent, warp specialised):
//
//   dB[e, n, k] = add[e, n, k] + sum over the rows m of group e of dC[m, n] * A[m, k]
//
// of bf16 or fp16 operands, or of e4m3 codes with a scale for each block of 128 rows of a column,
//
//   dB[e, n, k] = add + sum_t sc[t, n] * sa[t, k] * sum_{m in block t} dC[m, n] * A[m, k]
//
// The contraction runs over the rows, so both operands are MN-major as they lie and nothing is
// transposed.  Its length is the group's, known on the device only, and what follows the group's
// last row in memory belongs to the next one.  So the last stage of a group is special: its bytes
// are counted on a barrier of the CTA that loaded them, a fixer warp writes zeros over the rows
// behind the group's end in both operands (a NaN there would survive a zero in one), and hands the
// stage to the MMA thread; MMA steps that hold no row of the group are not issued.
//
// Sums: a chunk of rows accumulates in TMEM (fp8: the 128 rows of a scale block; 16-bit operands:
// CHUNK rows), and the epilogue warps add the chunks into fp32 registers, scaled by sc[n] * sa[k].
// The tensor core's own additions do not round to nearest; chunks keep them few (see CHUNK).
// Two chunks are in TMEM at a time, so that the MMAs of the next run meanwhile.
//
// Roles (12 warps): warp 0 TMA producer; warp 1 TMEM owner and, in CTA 0 of a pair, the MMA thread;
// warp 2 fixer; warps 4-11 epilogue (TMEM lanes 32 * (w % 4)..: columns n of dC; half of the tile's
// columns k each).
#include <atomic>
#include "expert_ops.cuh"
#include "ptx.cuh"

namespace bsfp8 {
namespace wg {

constexpr int THREADS = 384;
constexpr int EPI_WARP0 = 4;
constexpr int BN = 256;  // columns k of a tile
constexpr uint32_t TMEM_COLS = 512;

template <bool FP8_, int CG_, int STAGES_, int CHUNK_>
struct Cfg {
  static constexpr bool FP8 = FP8_;
  static constexpr int CG = CG_;
  static constexpr int BM = 128 * CG;             // columns n of a tile
  static constexpr int ROWS = FP8 ? 128 : 64;     // rows of the operands in a stage
  static constexpr int STEP = ROWS / 4;           // rows of an MMA (K = 32 or 16)
  static constexpr int CHUNK = FP8 ? 1 : CHUNK_;  // stages that accumulate in TMEM
  static constexpr int STAGES = STAGES_;
  static constexpr int BOX_COLS = FP8 ? 128 : 64;  // columns of a box: 128 bytes
  static constexpr uint32_t BOX = ROWS * 128;
  static constexpr int M_BOXES = 128 / BOX_COLS;         // of dC per CTA
  static constexpr int N_BOXES = BN / CG / BOX_COLS;     // of A per CTA
  static constexpr uint32_t STAGE = (M_BOXES + N_BOXES) * BOX;
  static constexpr uint32_t STEP_BYTES = STEP * 128;
  static constexpr uint32_t IDESC =
      (FP8 ? idesc_f8f6f4_e4m3(BM, BN) : idesc_f16_f32(BM, BN)) | IDESC_A_MN | IDESC_B_MN;
  // scales of a chunk's 128 columns k, per epilogue warp: fetched two chunks ahead
  static constexpr int SA_SLOTS = 4;
  static constexpr uint32_t SMEM_SA = STAGES * STAGE;
  static constexpr uint32_t SMEM_CTL = SMEM_SA + (FP8 ? 8 * SA_SLOTS * 128 * 4 : 0);
};

template <class C>
struct Ctl {
  uint64_t full[C::STAGES];
  uint64_t empty[C::STAGES];
  uint64_t tail[C::STAGES];       // the last stage of a group: this CTA's bytes
  uint64_t peer_tail[C::STAGES];  // leader: the peer's fixer is done with the stage
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int valid;
};

template <class C>
constexpr uint32_t smem_bytes() {
  return C::SMEM_CTL + sizeof(Ctl<C>) + 1024;  // + alignment slack
}

// Tiles are numbered expert by expert, inside one in bands of 8 column tiles of dC, whose columns
// of dC and A stay in L2 while the band's tiles are in flight.  An expert without rows has tiles
// too: its gradient is written.
struct Tile {
  int e, n0, k0;
  int64_t r0;
  int rows;
};

template <class C>
__device__ __forceinline__ Tile tile_at(const WgradArgs& a, int64_t t) {
  constexpr int BAND = 8;
  const int nt = (a.N + C::BM - 1) / C::BM, kt = (a.K + BN - 1) / BN;
  const int64_t per = (int64_t)nt * kt;
  Tile x;
  x.e = (int)(t / per);
  const int64_t local = t - x.e * per;
  const int band = (int)(local / ((int64_t)BAND * kt));
  const int in_band = (int)(local - (int64_t)band * BAND * kt);
  const int high = nt - band * BAND < BAND ? nt - band * BAND : BAND;
  x.n0 = (band * BAND + in_band % high) * C::BM;
  x.k0 = in_band / high * BN;
  x.r0 = a.offsets[x.e];
  x.rows = (int)(a.offsets[x.e + 1] - x.r0);
  return x;
}

__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Eight columns of a row of dB, `left` of which are the matrix's (8 or more: all).
template <int OUT>
__device__ __forceinline__ void store8(const WgradArgs& a, int64_t at, const float2* v,
                                       bool wide, uint64_t pol) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = v[j].x;
    f[2 * j + 1] = v[j].y;
  }
  if constexpr (OUT == GRAD_FP32) {
    if (a.add) {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(a.add) + at);
      const float4 x = s[0], y = s[1];
      f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
      f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(f[j]);
    float* d = static_cast<float*>(a.dB) + at;
    if (wide) {
      st_global_v8_hint(d, w, pol);
    } else {
      st_global_v4_hint(d, w[0], w[1], w[2], w[3], pol);
      st_global_v4_hint(d + 4, w[4], w[5], w[6], w[7], pol);
    }
  } else {
    if (a.add) {
      const uint4 s = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.add) + at);
      const uint32_t w[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (OUT == GRAD_BF16) {
          f[2 * j] += __uint_as_float(w[j] << 16);
          f[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
        } else {
          float lo, hi;
          asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
              "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
              : "=f"(lo), "=f"(hi)
              : "r"(w[j]));
          f[2 * j] += lo;
          f[2 * j + 1] += hi;
        }
      }
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = OUT == GRAD_BF16 ? pack_bf16x2(f[2 * j], f[2 * j + 1])
                              : pack_f16x2(f[2 * j], f[2 * j + 1]);
    st_global_v4_hint(static_cast<uint16_t*>(a.dB) + at, w[0], w[1], w[2], w[3], pol);
  }
}

template <class C, int OUT>
__global__ void __launch_bounds__(THREADS, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmA,
             const WgradArgs args, const int64_t total_tiles) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl<C>* ctl = reinterpret_cast<Ctl<C>*>(smem + C::SMEM_CTL);
  volatile int* abort = &ctl->abort;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = C::CG == 2 ? cluster_ctarank() : 0;
  const int64_t tile0 = blockIdx.x / C::CG;
  const int64_t tile_stride = gridDim.x / C::CG;

  if (warp == 0) {
    int64_t unused;
    const int status = check_groups<1>(args.offsets, nullptr, args.E, args.E, args.M_total, unused);
    if (lane == 0) {
      ctl->valid = status == 0;
      ctl->abort = 0;
      if (status && blockIdx.x == 0) atomicCAS(args.err, 0, status);
    }
  }
  __syncthreads();
  if (!ctl->valid || tile0 >= total_tiles) return;  // both CTAs of a pair agree

  const uint32_t base = smem_u32(smem);
  auto full_bar = [&](int s) { return smem_u32(&ctl->full[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&ctl->empty[s]); };
  auto tail_bar = [&](int s) { return smem_u32(&ctl->tail[s]); };
  auto peer_bar = [&](int s) { return smem_u32(&ctl->peer_tail[s]); };
  auto tfull_bar = [&](int s) { return smem_u32(&ctl->tfull[s]); };
  auto tempty_bar = [&](int s) { return smem_u32(&ctl->tempty[s]); };
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmC);
    tma_prefetch_desc(&tmA);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);   // the leader's producer (+ both CTAs' bytes), or its fixer
      mbar_init(empty_bar(s), 1);  // one commit
      mbar_init(tail_bar(s), 1);   // the producer (+ this CTA's bytes)
      mbar_init(peer_bar(s), 1);   // the peer's fixer
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull_bar(s), 1);           // one commit
      mbar_init(tempty_bar(s), 8 * C::CG);  // every epilogue warp of the pair
    }
    mbar_init(smem_u32(&ctl->mma_done), 1);
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc<C::CG>(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish<C::CG>();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C::CG == 2) cluster_sync();  // the peer's barriers before any use
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ------------------------------- TMA producer -------------------------------
      const uint64_t pol = l2_policy_evict_normal();
      uint32_t stage = 0, phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int64_t t = tile0; ok && t < total_tiles; t += tile_stride) {
        const Tile x = tile_at<C>(args, t);
        const int col_m = x.n0 + 128 * rank, col_n = x.k0 + (BN / C::CG) * rank;
        for (int r = 0; r < x.rows; r += C::ROWS) {
          if (!mbar_wait_sleep(empty_bar(stage), phase ^ 1, abort)) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          const uint32_t m = base + stage * C::STAGE, n = m + C::M_BOXES * C::BOX;
          const int32_t row = (int32_t)(x.r0 + r);
          if (C::CG == 1 || r + C::ROWS > x.rows) {
            // counted in this CTA: the fixer comes first where the group ends inside
            const uint32_t bar = r + C::ROWS > x.rows ? tail_bar(stage) : full_bar(stage);
            mbar_arrive_expect_tx(bar, C::STAGE);
            for (int i = 0; i < C::M_BOXES; ++i)
              tma_load_2d_hint(m + i * C::BOX, &tmC, col_m + i * C::BOX_COLS, row, bar, pol);
            for (int i = 0; i < C::N_BOXES; ++i)
              tma_load_2d_hint(n + i * C::BOX, &tmA, col_n + i * C::BOX_COLS, row, bar, pol);
          } else {
            // both CTAs' bytes are counted on the leader's barrier
            const uint32_t bar = mapa_shared(full_bar(stage), 0);
            if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * C::STAGE);
            for (int i = 0; i < C::M_BOXES; ++i)
              tma_load_2d_pair_hint(m + i * C::BOX, &tmC, col_m + i * C::BOX_COLS, row, bar, pol);
            for (int i = 0; i < C::N_BOXES; ++i)
              tma_load_2d_pair_hint(n + i * C::BOX, &tmA, col_n + i * C::BOX_COLS, row, bar, pol);
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
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // -------------------------------- MMA thread --------------------------------
      const uint32_t idesc = C::IDESC | (!C::FP8 && args.bf16 ? IDESC_BF16 : 0u);
      const uint64_t mdesc0 = mnmajor_sw128_desc(base, C::BOX);
      const uint64_t ndesc0 = mnmajor_sw128_desc(base + C::M_BOXES * C::BOX, C::BOX);
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = tile0; ok && t < total_tiles; t += tile_stride) {
        const Tile x = tile_at<C>(args, t);
        int in_chunk = 0;
        for (int r = 0; r < x.rows; r += C::ROWS) {
          if (!mbar_wait(full_bar(stage), phase, abort) ||
              (in_chunk == 0 && !mbar_wait(tempty_bar(acc), acc_phase ^ 1, abort))) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + acc * BN;
          const uint64_t mdesc = mdesc0 + ((stage * C::STAGE) >> 4);
          const uint64_t ndesc = ndesc0 + ((stage * C::STAGE) >> 4);
          const int steps = x.rows - r >= C::ROWS ? 4 : (x.rows - r + C::STEP - 1) / C::STEP;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k < steps) {
              const uint64_t go = (uint64_t)(k * C::STEP_BYTES) >> 4;
              if constexpr (C::FP8)
                umma_f8f6f4<C::CG>(d, mdesc + go, ndesc + go, idesc, (in_chunk | k) > 0);
              else
                umma_f16<C::CG>(d, mdesc + go, ndesc + go, idesc, (in_chunk | k) > 0);
            }
          }
          if constexpr (C::CG == 1) umma_commit(empty_bar(stage));
          else umma_commit_pair(empty_bar(stage), 0x3);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
          if (++in_chunk == C::CHUNK || r + C::ROWS >= x.rows) {
            if constexpr (C::CG == 1) umma_commit(tfull_bar(acc));
            else umma_commit_pair(tfull_bar(acc), 0x3);
            in_chunk = 0;
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
          }
        }
      }
      // every MMA has finished before TMEM is released
      if constexpr (C::CG == 1) umma_commit(smem_u32(&ctl->mma_done));
      else umma_commit_pair(smem_u32(&ctl->mma_done), 0x1);
      if (!mbar_wait_timed(smem_u32(&ctl->mma_done), 0)) give_up(args.err, abort);
    } else if (warp == 2) {
      // ----------------------------------- fixer -----------------------------------
      // Of the last stage of each group whose rows do not fill it: zeros from the group's end to
      // the end of the MMA step that holds it (whole 128-byte lines, whatever the swizzle).
      uint32_t stage = 0;
      uint32_t seen = 0;  // parity of every stage's tail barrier, a bit each
      for (int64_t t = tile0; t < total_tiles; t += tile_stride) {
        const Tile x = tile_at<C>(args, t);
        const int stages = (x.rows + C::ROWS - 1) / C::ROWS;
        const int left = x.rows % C::ROWS;
        const uint32_t last = (stage + stages + C::STAGES - 1) % C::STAGES;
        stage = (stage + stages) % C::STAGES;
        if (left == 0) continue;
        const uint32_t parity = (seen >> last) & 1;
        seen ^= 1u << last;
        if (!__all_sync(0xffffffffu, mbar_wait_sleep(tail_bar(last), parity, abort))) {
          if (lane == 0) give_up(args.err, abort);
          break;
        }
        const int end = (left + C::STEP - 1) / C::STEP * C::STEP;
        for (int b = 0; b < C::M_BOXES + C::N_BOXES; ++b) {
          uint4* lines = reinterpret_cast<uint4*>(smem + last * C::STAGE + b * C::BOX);
          for (int i = left * 8 + lane; i < end * 8; i += 32) lines[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (rank == 1) {
            mbar_arrive_release_cluster(mapa_shared(peer_bar(last), 0));
          } else {
            if (C::CG == 2 && !mbar_wait_cluster(peer_bar(last), parity, abort))
              give_up(args.err, abort);
            else
              mbar_arrive(full_bar(last));
          }
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    // --------------------------------- epilogue ---------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const uint32_t w = warp - EPI_WARP0;
    const uint32_t quarter = warp & 3, half = w >> 2;
    const uint64_t pol = l2_policy_evict_first();
    const bool wide = (reinterpret_cast<uintptr_t>(args.dB) & 31) == 0 && args.K % 8 == 0;
    const uint32_t taddr0 = tmem_base + ((quarter * 32) << 16) + half * 128;
    uint32_t acc = 0, acc_phase = 0;
    bool ok = true;

    // fp8: this warp's column scales go through SA_SLOTS slots of shared memory, a chunk each,
    // and this lane's row scale through registers; both are fetched two chunks ahead, those of a
    // tile's first two before the tile before it is stored.
    float* sa_slots = reinterpret_cast<float*>(smem + C::SMEM_SA) + w * C::SA_SLOTS * 128;
    uint32_t slot = 0;  // of the chunk that is added next
    float sc_0 = 0.0f, sc_1 = 0.0f;
    auto chunks_of = [&](const Tile& x) {
      return (x.rows + C::ROWS * C::CHUNK - 1) / (C::ROWS * C::CHUNK);
    };
    auto fetch = [&](const Tile& x, int chunk, uint32_t to) {
      float sc = 0.0f;
      if (chunk < chunks_of(x)) {
        const int64_t s = x.r0 / 128 + x.e + chunk;
        const int n = x.n0 + 128 * (int)rank + (int)quarter * 32 + (int)lane;
        const int k = x.k0 + (int)half * 128 + 4 * (int)lane;
        const bool in = x.k0 + (int)half * 128 < args.K;  // K is a multiple of 128
        cp_async_16(smem_u32(sa_slots + (to % C::SA_SLOTS) * 128 + 4 * lane),
                    args.a_scales + s * args.K + (in ? k : 0), in ? 16 : 0);
        if (n < args.N) sc = args.dc_scales[s * args.N + n];
      }
      cp_async_commit();
      return sc;
    };

    Tile x = {};
    if (tile0 < total_tiles) {
      x = tile_at<C>(args, tile0);
      if constexpr (C::FP8) {
        sc_0 = fetch(x, 0, slot);
        sc_1 = fetch(x, 1, slot + 1);
      }
    }
    for (int64_t t = tile0; ok && t < total_tiles; t += tile_stride) {
      float2 sum[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) sum[j] = make_float2(0.0f, 0.0f);
      const int chunks = chunks_of(x);
      for (int c = 0; c < chunks; ++c) {
        float sc = 1.0f;
        if constexpr (C::FP8) {
          sc = sc_0;
          sc_0 = sc_1;
          sc_1 = fetch(x, c + 2, slot + 2);
          cp_async_wait_group<2>();
          __syncwarp();
        }
        if (!__all_sync(0xffffffffu, mbar_wait(tfull_bar(acc), acc_phase, abort))) {
          if (lane == 0) give_up(args.err, abort);
          ok = false;
          break;
        }
        tc_fence_after();
        const float2 sc2 = make_float2(sc, sc);
        const float4* sa = reinterpret_cast<const float4*>(sa_slots + (slot % C::SA_SLOTS) * 128);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[64];
          tmem_ld_32x32b_x64(taddr0 + acc * BN + 64 * h, p);
          tmem_ld_wait();
          if (h == 1) {  // TMEM is read: the MMA thread may have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
              mbar_arrive_cluster_or_local<C::CG>(C::CG == 2 ? mapa_shared(tempty_bar(acc), 0)
                                                             : tempty_bar(acc));
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float2 a = make_float2(__uint_as_float(p[2 * j]), __uint_as_float(p[2 * j + 1]));
            float2 b = make_float2(__uint_as_float(p[2 * j + 2]), __uint_as_float(p[2 * j + 3]));
            if constexpr (C::FP8) {
              const float4 s = sa[16 * h + j / 2];
              a = mul_f32x2(a, make_float2(s.x, s.y));
              b = mul_f32x2(b, make_float2(s.z, s.w));
            }
            sum[32 * h + j] = __ffma2_rn(sc2, a, sum[32 * h + j]);
            sum[32 * h + j + 1] = __ffma2_rn(sc2, b, sum[32 * h + j + 1]);
          }
        }
        ++slot;
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok) break;
      const Tile now = x;
      if (t + tile_stride < total_tiles) {
        x = tile_at<C>(args, t + tile_stride);
        if constexpr (C::FP8) {
          // a tile of fewer than two chunks left later slots fetched for nothing: start behind
          sc_0 = fetch(x, 0, slot);
          sc_1 = fetch(x, 1, slot + 1);
        }
      }
      const int n = now.n0 + 128 * (int)rank + (int)quarter * 32 + (int)lane;
      const int k0 = now.k0 + (int)half * 128;
      if (n < args.N) {
        const int64_t at = ((int64_t)now.e * args.N + n) * args.K + k0;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (k0 + 8 * j < args.K) store8<OUT>(args, at + 8 * j, sum + 4 * j, wide, pol);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // the pair's MMAs and remote arrivals are finished before either CTA frees TMEM or exits
  if constexpr (C::CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<C::CG>(tmem_base, TMEM_COLS);
  }
}

template <class C, int OUT>
cudaError_t launch(const WgradArgs& args, int num_sms, cudaStream_t stream) {
  static_assert(smem_bytes<C>() <= 227 * 1024, "shared memory per CTA");
  CUtensorMap tmC, tmA;
  // with no rows nothing is loaded; a map still needs a row
  const uint64_t rows = args.M_total > 0 ? (uint64_t)args.M_total : 1;
  const uint64_t c_dims[2] = {(uint64_t)args.N, rows}, a_dims[2] = {(uint64_t)args.K, rows};
  if (!encode_swizzled(&tmC, C::FP8, args.M_total > 0 ? args.dC : args.dB, 2, c_dims, C::ROWS) ||
      !encode_swizzled(&tmA, C::FP8, args.M_total > 0 ? args.A : args.dB, 2, a_dims, C::ROWS))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];  // per device; several host threads may launch
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(wgrad_kernel<C, OUT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes<C>());
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  const int64_t tiles = (int64_t)args.E * ((args.N + C::BM - 1) / C::BM) * ((args.K + BN - 1) / BN);
  const int64_t units = num_sms / C::CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < units ? tiles : units) * C::CG));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes<C>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, wgrad_kernel<C, OUT>, tmC, tmA, args, tiles);
}

template <class C>
cudaError_t by_type(const WgradArgs& a, int num_sms, cudaStream_t stream) {
  switch (a.out_type) {
    case GRAD_BF16: return launch<C, GRAD_BF16>(a, num_sms, stream);
    case GRAD_FP16: return launch<C, GRAD_FP16>(a, num_sms, stream);
    default: return launch<C, GRAD_FP32>(a, num_sms, stream);
  }
}

}  // namespace wg

cudaError_t launch_wgrad(const WgradArgs& a, int num_sms, cudaStream_t stream) {
  return a.fp8 ? wg::by_type<wg::Cfg<true, 2, 6, 1>>(a, num_sms, stream)
               : wg::by_type<wg::Cfg<false, 2, 6, 8>>(a, num_sms, stream);
}

}  // namespace bsfp8
