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
// 512 rows), and the epilogue warps add the chunks into fp32 registers, scaled by sc[n] * sa[k].
// The tensor core's additions do not round to nearest, and their errors add up: of 65536 rows in
// one chunk the sum is off by 7.6e-5 of its norm, in chunks of 2048 by 2.1e-6, of 512 by 5e-7 (some 230
// rows in one chunk 3.2e-7, where a sum that rounds is off by 1.4e-7); chunks of 512 cost 3 % of the
// time of one.  Two chunks are in TMEM at a time, so that the MMAs of the next run meanwhile.
//
// What bounds it: 16-bit, the tensor core and the operands' way from L2 (65536 rows, 2048 x 4608:
// 702 us, 1762 TFLOP/s with 144 tiles for 76 pairs; the loads alone 525) or, with few rows per
// expert, the gradients' bytes (16384 rows over 64 experts of 2048 x 7168 to fp32: 612 us, 6.6
// TB/s).  8 bits, the sums' way out of TMEM: every block of 128 rows has its own scales, so its sums
// are handed to the epilogue after 512 clocks of MMA, and half of TMEM is taken until they are read
// and their 2 operations per element under way (the same rows: 589 us, 2099 TFLOP/s; if 256 rows
// made a block 438, without the scales' products 511, the loads alone 333).
//
// What made it so: a stage's one commit is the hand-over's too (8 bits, 16 groups of 2048 rows, 2048 x
// 7168: 594 -> 576 us), and the sums go out by TMA (565).  The scales land with the operands, counted
// on their barrier (65536 rows, 2048 x 4608: read from global memory two blocks ahead, the epilogue
// waited for them, 826); a warp reads TMEM as 16 x 256-bit pieces, of which a thread gets 4 rows x 32
// columns, 36 scales, and not a row of 128 columns, 129 (shared memory is what the MMA is fed from:
// 740 -> 646); the pieces are double-buffered, with registers to hold them (589); the 16-bit roles
// that wait beside the epilogue sleep in their barriers (880 -> 785, then stages of 128 rows, 702).
// Four stages: with six the loads of operands run so far ahead that they stand in the way of the
// gradients' stores (16384 rows over 64 experts: 745 -> 617).
//
// Roles (12 warps): warp 0 TMA producer; warp 1 TMEM owner and, in CTA 0 of a pair, the MMA thread;
// warp 2 fixer; warps 4-11 epilogue (TMEM lanes 32 * (w % 4)..: columns n of dC; half of the tile's
// columns k each).
#include "expert_ops.cuh"
#include "ptx.cuh"

namespace bsfp8 {
namespace wg {

constexpr int THREADS = 384;
constexpr int EPI_WARP0 = 4;
constexpr int BN = 256;  // columns k of a tile
constexpr uint32_t TMEM_COLS = 512;

// ROWS: of the operands in a stage.  SPLIT: pairs, in one cluster, that share a tile's rows, each
// cluster one tile.  STAGED: the gradients are stored by TMA, out of shared memory.
template <bool FP8_, int ROWS_, int STAGES_, bool STAGED_, int SPLIT_ = 1>
struct Cfg {
  static constexpr bool FP8 = FP8_;
  static constexpr int CG = 2;
  static constexpr int SPLIT = SPLIT_;
  static constexpr int BM = 128 * CG;  // columns n of a tile
  static constexpr int ROWS = ROWS_;
  static constexpr int STEP = FP8 ? 32 : 16;  // rows of an MMA
  static constexpr int STEPS = ROWS / STEP;
  static constexpr int CHUNK = (FP8 ? 128 : 512) / ROWS;  // stages that accumulate in TMEM
  static constexpr int STAGES = STAGES_;
  static constexpr int BOX_COLS = FP8 ? 128 : 64;  // columns of a box: 128 bytes
  static constexpr uint32_t BOX = ROWS * 128;
  static constexpr int M_BOXES = 128 / BOX_COLS;         // of dC per CTA
  static constexpr int N_BOXES = BN / CG / BOX_COLS;     // of A per CTA
  static constexpr uint32_t STAGE = (M_BOXES + N_BOXES) * BOX;
  static constexpr uint32_t STAGE_TX = STAGE + (FP8 ? (BN + 128) * 4 : 0);  // and its scales
  static constexpr uint32_t STEP_BYTES = STEP * 128;
  // registers of the role warps and of the epilogue warps, of the 168 each is launched with
  static constexpr int ROLE_REGS = 40;
  static constexpr int SUM_REGS = 232;
  // a split tile's part of the sums, 128 x 256 in fp32, takes the operands' ring when that is done
  static_assert(SPLIT == 1 || 128 * BN * 4 <= STAGES * STAGE, "part");
  static_assert(4 * ROLE_REGS + 8 * SUM_REGS <= 12 * 168, "the launch's registers");
  static constexpr uint32_t IDESC =
      (FP8 ? idesc_f8f6f4_e4m3(BM, BN) : idesc_f16_f32(BM, BN)) | IDESC_A_MN | IDESC_B_MN;
  // fp8: slots of a stage's scales, [256 columns k | 128 columns n] (see the producer)
  static constexpr int SLOTS = 2 * STAGES;
  static constexpr uint32_t SLOT = (BN + 128) * 4;
  // where a warp of the epilogue puts 32 rows of 128 bytes for TMA to store: twice, where it fits
  static constexpr uint32_t OUT_BOX = 4096;
  static constexpr int OUT_BOXES =
      !STAGED_ ? 0 : STAGES * STAGE + 16 * OUT_BOX + (FP8 ? SLOTS * SLOT : 0) <= 224 * 1024 ? 2 : 1;
  static constexpr uint32_t SMEM_OUT = STAGES * STAGE;
  static constexpr uint32_t SMEM_SF = SMEM_OUT + 8 * OUT_BOXES * OUT_BOX;
  static constexpr uint32_t SMEM_CTL = SMEM_SF + (FP8 ? SLOTS * SLOT : 0);
  static_assert(SPLIT == 1 || !STAGED_, "a split tile's stripes are stored by their threads");
  static_assert(!FP8 || SLOTS >= STAGES + 2, "a slot is read to the end before it is filled again");
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
  uint32_t issued;  // stages that this CTA's producer has sent for
  int abort;
  int valid;
};

template <class C>
constexpr uint32_t smem_bytes() {
  return C::SMEM_CTL + sizeof(Ctl<C>) + 1024;  // + alignment slack
}

// Groups of rows may end before M_total: offsets[0] == 0 <= offsets[1] <= .. <= offsets[E] <=
// M_total.  One full warp checks them; every lane gets the status (0 or a device error code).
__device__ __forceinline__ int check_offsets(const int32_t* off, int E, int64_t M_total) {
  int good = 1;
  for (int e = (int)lane_id(); e < E; e += 32) {
    const int a = off[e], b = off[e + 1];
    if (a < 0 || b < a || b > M_total || (e == 0 && a != 0)) good = 0;
  }
  return __all_sync(0xffffffffu, good) ? 0 : DEV_BAD_OFFSETS;
}

// Tiles are numbered expert by expert, inside one in bands of 8 column tiles of dC, whose columns
// of dC and A stay in L2 while the band's tiles are in flight.  An expert without rows has tiles
// too: its gradient is written.  A role walks the tiles `stride` apart; the walk is a few integers
// (the roles' warps have few registers).
struct Shape {
  uint32_t experts, nt, kt;  // tiles per side of an expert's matrix
};

struct Walk {
  uint32_t e = 0, local;
  __device__ explicit Walk(uint32_t first) : local(first) {}
  __device__ bool inside(const Shape& s) {  // and to the tile's expert
    const uint32_t per = s.nt * s.kt;
    while (local >= per && e < s.experts) {
      local -= per;
      ++e;
    }
    return e < s.experts;
  }
  // The rows of the tile's group that a pair takes: all, or of SPLIT parts one, whole blocks of 128.
  template <int SPLIT>
  __device__ void rows(const WgradArgs& a, uint32_t part, int& begin, int& end) const {
    const int all = a.offsets[e + 1] - a.offsets[e];
    begin = 0;
    end = all;
    if constexpr (SPLIT > 1) {
      const int64_t blocks = (all + 127) / 128;
      begin = (int)(blocks * part / SPLIT) * 128;
      if (part + 1 < SPLIT) end = (int)(blocks * (part + 1) / SPLIT) * 128;
    }
  }
  template <int BM>
  __device__ void corner(const Shape& s, int& n0, int& k0) const {
    constexpr uint32_t BAND = 8;
    const uint32_t band = local / (BAND * s.kt), in_band = local - band * BAND * s.kt;
    const uint32_t high = s.nt - band * BAND < BAND ? s.nt - band * BAND : BAND;
    n0 = (int)((band * BAND + in_band % high) * BM);
    k0 = (int)(in_band / high * BN);
  }
};

__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// v[j] of lane 4 r + q becomes v[q] of lane 4 r + j.
__device__ __forceinline__ void quad_transpose(float2 (&v)[4], uint32_t lane) {
#pragma unroll
  for (int d = 1; d <= 2; d *= 2) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & d) continue;
      // the lower lane gives its v[j + d] for the upper one's v[j]
      float2 out = up ? v[j] : v[j + d];
      out.x = __shfl_xor_sync(0xffffffffu, out.x, d);
      out.y = __shfl_xor_sync(0xffffffffu, out.y, d);
      if (up) v[j] = out;
      else v[j + d] = out;
    }
  }
}

// Eight columns of a row of a 16-bit add; not the read-only path, as add may be dB.
template <int OUT>
__device__ __forceinline__ void load8(const void* add, int64_t at, float2 (&v)[4]) {
  uint32_t w[4];
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(static_cast<const uint16_t*>(add) + at));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (OUT == GRAD_BF16) {
      v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    } else {
      asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
          "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
          : "=f"(v[j].x), "=f"(v[j].y)
          : "r"(w[j]));
    }
  }
}

// The same of words.
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[4], uint32_t lane) {
#pragma unroll
  for (int d = 1; d <= 2; d *= 2) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & d) continue;
      const uint32_t out = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + d], d);
      if (up) v[j] = out;
      else v[j + d] = out;
    }
  }
}

// Pairs of columns 8 j + 2 (lane % 4).. of a row, j < 4, exchanged between the four lanes that hold
// the row and stored, eight columns 8 (lane % 4).. by each; 16-bit values are rounded first.
template <int OUT>
__device__ __forceinline__ void store_row(void* dB, int64_t at, float2 (&v)[4], bool in, bool wide,
                                          uint32_t lane, uint64_t pol) {
  if constexpr (OUT == GRAD_FP32) {
    quad_transpose(v, lane);
    if (!in) return;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[2 * j] = __float_as_uint(v[j].x);
      w[2 * j + 1] = __float_as_uint(v[j].y);
    }
    float* d = static_cast<float*>(dB) + at;
    if (wide) {
      st_global_v8_hint(d, w, pol);
    } else {
      st_global_v4_hint(d, w[0], w[1], w[2], w[3], pol);
      st_global_v4_hint(d + 4, w[4], w[5], w[6], w[7], pol);
    }
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = OUT == GRAD_BF16 ? pack_bf16x2(v[j].x, v[j].y) : pack_f16x2(v[j].x, v[j].y);
    quad_transpose(w, lane);
    if (in) st_global_v4_hint(static_cast<uint16_t*>(dB) + at, w[0], w[1], w[2], w[3], pol);
  }
}

// A box for TMA to store, of a warp's 32 rows and their columns 32 g.. (fp32) or 64 g..: 128 bytes of
// each row, 16-byte chunk c of row r at c ^ r % 8.  The lanes of odd rows begin with other columns,
// so that no two of a half-warp meet in a bank.
template <int OUT>
__device__ __forceinline__ void fill_box(uint32_t box, const float2 (&sum)[4][4][4], int g, uint32_t lane) {
  const uint32_t r = lane / 4, q = lane % 4;
  const uint32_t at = box + r * 128;
  if constexpr (OUT == GRAD_FP32) {
    const bool odd = r % 2;
    const uint32_t chunk = (q / 2) ^ r ^ (odd ? 4 : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float2 v = odd ? sum[i][g][s ^ 2] : sum[i][g][s];
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at + i * 1024 + ((chunk ^ (2 * s)) << 4) + 8 * (q % 2)),
                     "f"(v.x), "f"(v.y)
                     : "memory");
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float2 v = sum[i][2 * g + c / 4][c % 4];
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + i * 1024 + ((r ^ c) << 4) + 4 * q),
                     "r"(OUT == GRAD_BF16 ? pack_bf16x2(v.x, v.y) : pack_f16x2(v.x, v.y))
                     : "memory");
      }
    }
  }
}

template <class C, int OUT>
__global__ void __launch_bounds__(THREADS, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmA,
             const __grid_constant__ CUtensorMap tmSC, const __grid_constant__ CUtensorMap tmSA,
             const __grid_constant__ CUtensorMap tmD,  // dB, to be stored
             const WgradArgs args, const Shape shape) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl<C>* ctl = reinterpret_cast<Ctl<C>*>(smem + C::SMEM_CTL);
  volatile int* abort = &ctl->abort;
  volatile uint32_t* sent = &ctl->issued;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  // of the CTA in its pair, its pair's leader in the cluster, and the pair's share of a split tile
  const uint32_t cta = cluster_ctarank();
  const uint32_t rank = cta % C::CG, leader = cta - rank, part = cta / C::CG;
  const uint16_t both = (uint16_t)(0x3 << leader);
  // the grid has no more clusters than there are tiles (as many, where they are split)
  const uint32_t tile0 = blockIdx.x / (C::CG * C::SPLIT);
  const uint32_t tile_stride = gridDim.x / (C::CG * C::SPLIT);

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
    ctl->abort = 0;
    ctl->issued = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc<C::CG>(smem_u32(&ctl->tmem_base), TMEM_COLS);
    tmem_relinquish<C::CG>();
    launch_dependents();
  }
  wait_for_previous();
  if (warp == 2) {
    const int status = check_offsets(args.offsets, args.E, args.M_total);
    if (lane == 0) {
      ctl->valid = status == 0;
      if (status && blockIdx.x == 0) atomicCAS(args.err, 0, status);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers before any use
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const bool valid = ctl->valid;  // both CTAs of a pair agree

  // (of a split tile, every warp is in the cluster's barrier between the parts and their sum)
  if (!valid) {
    if constexpr (C::SPLIT > 1) cluster_sync();
  } else if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::ROLE_REGS));
    if (warp == 0 && lane == 0) {
      // ------------------------------- TMA producer -------------------------------
      // fp8: a stage's scales go into a ring of their own, which no barrier frees: the MMAs that
      // this stage waits for (STAGES blocks ago) began when every epilogue warp had read the
      // partial sums, and before them the scales, of two blocks earlier.
      const uint64_t pol = l2_policy_evict_normal();
      uint32_t stage = 0, phase = 0, slot = 0;
      int64_t issued = 0;
      bool ok = true;
      for (Walk t(tile0); ok && t.inside(shape); t.local += tile_stride) {
        int begin, rows;  // (of the group: up to the pair's last)
        t.rows<C::SPLIT>(args, part, begin, rows);
        const int r0 = args.offsets[t.e];
        int n0, k0;
        t.corner<C::BM>(shape, n0, k0);
        const int col_m = n0 + 128 * rank, col_n = k0 + (BN / C::CG) * rank;
        for (int r = begin; r < rows; r += C::ROWS) {
          if (!mbar_wait_sleep(empty_bar(stage), phase ^ 1, abort)) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          const uint32_t m = base + stage * C::STAGE, n = m + C::M_BOXES * C::BOX;
          const int32_t row = r0 + r;
          const int32_t at = r0 / 128 + (int)t.e + r / 128;  // fp8: its scales' row
          const uint32_t dst = base + C::SMEM_SF + slot * C::SLOT;
          if (r + C::ROWS > rows) {
            // the group ends inside: counted in this CTA, whose fixer comes first
            const uint32_t bar = tail_bar(stage);
            mbar_arrive_expect_tx(bar, C::STAGE_TX);
#pragma unroll
            for (int i = 0; i < C::M_BOXES; ++i)
              tma_load_2d_hint(m + i * C::BOX, &tmC, col_m + i * C::BOX_COLS, row, bar, pol);
#pragma unroll
            for (int i = 0; i < C::N_BOXES; ++i)
              tma_load_2d_hint(n + i * C::BOX, &tmA, col_n + i * C::BOX_COLS, row, bar, pol);
            if constexpr (C::FP8) {
              tma_load_2d_hint(dst, &tmSA, k0, at, bar, pol);
              tma_load_2d_hint(dst + BN * 4, &tmSC, col_m, at, bar, pol);
            }
          } else {
            // both CTAs' bytes are counted on the leader's barrier
            const uint32_t bar = mapa_shared(full_bar(stage), leader);
            if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * C::STAGE_TX);
#pragma unroll
            for (int i = 0; i < C::M_BOXES; ++i)
              tma_load_2d_pair_hint(m + i * C::BOX, &tmC, col_m + i * C::BOX_COLS, row, bar, pol);
#pragma unroll
            for (int i = 0; i < C::N_BOXES; ++i)
              tma_load_2d_pair_hint(n + i * C::BOX, &tmA, col_n + i * C::BOX_COLS, row, bar, pol);
            if constexpr (C::FP8) {
              tma_load_2d_pair_hint(dst, &tmSA, k0, at, bar, pol);
              tma_load_2d_pair_hint(dst + BN * 4, &tmSC, col_m, at, bar, pol);
            }
          }
          if (++slot == C::SLOTS) slot = 0;
          *sent = (uint32_t)++issued;
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
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return C::FP8 ? mbar_wait(bar, parity, abort) : mbar_wait_sleep(bar, parity, abort);
      };
      for (Walk t(tile0); ok && t.inside(shape); t.local += tile_stride) {
        int begin, rows;
        t.rows<C::SPLIT>(args, part, begin, rows);
        int in_chunk = 0;
        for (int r = begin; r < rows; r += C::ROWS) {
          if (!wait(full_bar(stage), phase)) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          if (in_chunk == 0 && !wait(tempty_bar(acc), acc_phase ^ 1)) {
            give_up(args.err, abort);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + acc * BN;
          const uint64_t mdesc = mdesc0 + ((stage * C::STAGE) >> 4);
          const uint64_t ndesc = ndesc0 + ((stage * C::STAGE) >> 4);
          const int steps = rows - r >= C::ROWS ? C::STEPS : (rows - r + C::STEP - 1) / C::STEP;
#pragma unroll
          for (int k = 0; k < C::STEPS; ++k) {
            if (k < steps) {
              const uint64_t go = (uint64_t)(k * C::STEP_BYTES) >> 4;
              if constexpr (C::FP8)
                umma_f8f6f4<C::CG>(d, mdesc + go, ndesc + go, idesc, (in_chunk | k) > 0);
              else
                umma_f16<C::CG>(d, mdesc + go, ndesc + go, idesc, (in_chunk | k) > 0);
            }
          }
          umma_commit_pair(empty_bar(stage), both);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
          if (++in_chunk == C::CHUNK || r + C::ROWS >= rows) {
            if constexpr (!C::FP8) umma_commit_pair(tfull_bar(acc), both);
            in_chunk = 0;
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
          }
        }
      }
      // every MMA has finished before TMEM is released
      umma_commit_pair(smem_u32(&ctl->mma_done), (uint16_t)(1 << leader));
      if (!mbar_wait_timed(smem_u32(&ctl->mma_done), 0)) give_up(args.err, abort);
    } else if (warp == 2) {
      // ----------------------------------- fixer -----------------------------------
      // Of the last stage of each group whose rows do not fill it: zeros from the group's end to
      // the end of the MMA step that holds it (whole 128-byte lines, whatever the swizzle).
      uint32_t stage = 0;
      uint32_t seen = 0;  // parity of every stage's tail barrier, a bit each
      // Before a tail its whole group goes by, and every tile before it that had none: a wait has
      // run out when for its limit the producer has sent for nothing either.
      auto landed = [&](uint32_t bar, uint32_t parity) {
        uint32_t before = *sent;
        while (!mbar_wait_sleep(bar, parity, abort)) {
          const uint32_t now = *sent;
          if (*abort || now == before) return false;
          before = now;
        }
        return true;
      };
      for (Walk t(tile0); t.inside(shape); t.local += tile_stride) {
        int begin, rows;
        t.rows<C::SPLIT>(args, part, begin, rows);
        const int stages = (rows - begin + C::ROWS - 1) / C::ROWS;
        const int left = (rows - begin) % C::ROWS;
        const uint32_t last = (stage + stages + C::STAGES - 1) % C::STAGES;
        stage = (stage + stages) % C::STAGES;
        if (left == 0) continue;
        const uint32_t parity = (seen >> last) & 1;
        seen ^= 1u << last;
        if (!__all_sync(0xffffffffu, landed(tail_bar(last), parity))) {
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
            mbar_arrive_release_cluster(mapa_shared(peer_bar(last), leader));
          } else {
            if (!mbar_wait_cluster(peer_bar(last), parity, abort))
              give_up(args.err, abort);
            else
              mbar_arrive(full_bar(last));
          }
        }
        __syncwarp();
      }
    }
    __syncwarp();
    if constexpr (C::SPLIT > 1) cluster_sync();
  } else {
    // --------------------------------- epilogue ---------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SUM_REGS));
    const uint32_t quarter = warp & 3, half = (warp - EPI_WARP0) >> 2;
    const uint64_t pol = l2_policy_evict_first();
    const bool wide = (reinterpret_cast<uintptr_t>(args.dB) & 31) == 0 && args.K % 8 == 0;
    const uint32_t taddr0 = tmem_base + ((quarter * 32) << 16) + half * 128;
    uint32_t acc = 0, acc_phase = 0;
    bool ok = true;

    uint32_t slot = 0;
    // 16-bit chunks are long: the warps sleep, so as not to poll beside the MMA thread (8 bits: a
    // wake-up counts at each block; as there, 597 -> 588 us)
    auto wait = [&](uint32_t bar, uint32_t parity) {
      return C::FP8 ? mbar_wait(bar, parity, abort) : mbar_wait_sleep(bar, parity, abort);
    };
    const uint32_t tempty_0 = mapa_shared(tempty_bar(0), leader);
    const uint32_t tempty_1 = mapa_shared(tempty_bar(1), leader);
    for (Walk t(tile0); t.inside(shape); t.local += tile_stride) {
      int begin, rows, n0, k0;
      t.rows<C::SPLIT>(args, part, begin, rows);
      t.corner<C::BM>(shape, n0, k0);
      // Rows n of lanes lane / 4 + 8 i, columns 8 g + 2 (lane % 4) and the next.  The sums begin
      // with add, whose loads need no registers of their own here: fp32 pairs go where they
      // belong, of 16-bit values each lane reads 8 columns of a row, and four lanes exchange
      // theirs (as they do before dB is stored).
      n0 += 128 * (int)rank + (int)quarter * 32 + (int)lane / 4;
      k0 += (int)half * 128;
      const int k8 = k0 + 8 * (int)(lane % 4);
      float2 sum[4][4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[i][g][j] = make_float2(0.0f, 0.0f);
      if (args.add && part == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t row = ((int64_t)t.e * args.N + n0 + 8 * i) * args.K;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if constexpr (OUT == GRAD_FP32) {
              const float* p = static_cast<const float*>(args.add) + row + k0 + 32 * g + 2 * (lane % 4);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (n0 + 8 * i < args.N && k0 + 32 * g + 8 * j < args.K)
                  asm volatile("ld.global.v2.f32 {%0, %1}, [%2];"
                               : "=f"(sum[i][g][j].x), "=f"(sum[i][g][j].y)
                               : "l"(p + 8 * j));
            } else {
              if (n0 + 8 * i < args.N && k8 + 32 * g < args.K)
                load8<OUT>(args.add, row + k8 + 32 * g, sum[i][g]);
            }
          }
        }
        // The next tile's go into L2 meanwhile, a line at a time.  16-bit values are waited for by the
        // exchange (64 experts of 2048 x 7168, 256 rows each, bf16 added: 1319 -> 1058 us).  fp32
        // pairs are waited for by the first sums only: 8 bits gain by it where a tile takes long
        // enough to hide the lines (32 experts, 384 rows each 873 -> 735 us, 256 rows 627 -> 697), 16
        // bits lose (384 rows 643 -> 771, 1024 rows 825 -> 830).
        if (OUT != GRAD_FP32 || (C::FP8 && rows - begin >= 384)) {
          constexpr int SIZE = OUT == GRAD_FP32 ? 4 : 2;
          Walk next = t;
          next.local += tile_stride;
          if (next.inside(shape)) {
            int n, k;
            next.corner<C::BM>(shape, n, k);
            n += 128 * (int)rank + (int)quarter * 32 + (int)lane;
            k += (int)half * 128;
            const uint8_t* p = static_cast<const uint8_t*>(args.add) +
                               (((int64_t)next.e * args.N + n) * args.K + k) * SIZE;
#pragma unroll
            for (int c = 0; c < 128; c += 128 / SIZE)
              if (n < args.N && k + c < args.K) prefetch_l2(p + c * SIZE);
          }
        }
        if constexpr (OUT != GRAD_FP32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) quad_transpose(sum[i][g], lane);
        }
      }
      // A chunk's 32 rows x 128 columns come in pieces of 32 columns, one in flight while the one
      // before is added: the first of the next chunk too, so that the loads' latency is hidden but
      // at a tile's start.  One wait is for all: the MMAs began when the stage's scales had landed.
      // A lane that gives up goes through the motions to the tile's end, where all of them look.
      uint32_t p[2][2][16];
      auto load = [&](int q) {  // columns 32 q..
        tmem_ld_16x256b_x4(taddr0 + acc * BN + 32 * q, p[q % 2][0]);
        tmem_ld_16x256b_x4(taddr0 + (16 << 16) + acc * BN + 32 * q, p[q % 2][1]);
      };
      auto start = [&](uint32_t s) {  // fp8: a chunk is a stage, whose commit says so
        ok &= C::FP8 ? wait(empty_bar(s % C::STAGES), s / C::STAGES) : wait(tfull_bar(acc), acc_phase);
        __syncwarp();
        tc_fence_after();
        load(0);
      };
      if (rows > begin) start(slot);
      for (int r = begin; r < rows; r += C::ROWS * C::CHUNK) {
        float sc[4];
        float2 sa[4];
        const float* scales = reinterpret_cast<const float*>(smem + C::SMEM_SF + slot * C::SLOT);
        const float2* sa_at = reinterpret_cast<const float2*>(scales + half * 128) + lane % 4;
        if constexpr (C::FP8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[i] = scales[BN + quarter * 32 + lane / 4 + 8 * i];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (C::FP8) {
#pragma unroll
            for (int g = 0; g < 4; ++g) sa[g] = sa_at[16 * q + 4 * g];
          }
          tmem_ld_wait();
          if (q < 3) {
            load(q + 1);
          } else {  // TMEM is read: the MMA thread may have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_or_local<C::CG>(acc ? tempty_1 : tempty_0);
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            if (r + C::ROWS * C::CHUNK < rows) start((slot + 1) % C::SLOTS);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const uint32_t* w = &p[q % 2][i / 2][4 * g + 2 * (i % 2)];
              const float2 v = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
              float2& to = sum[i][q][g];
              if constexpr (C::FP8)
                to = __ffma2_rn(make_float2(sc[i], sc[i]), mul_f32x2(v, sa[g]), to);
              else
                to = __ffma2_rn(make_float2(1.0f, 1.0f), v, to);
            }
          }
        }
        if (++slot == C::SLOTS) slot = 0;
      }
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) give_up(args.err, abort);
        if constexpr (C::SPLIT > 1) cluster_sync();
        break;
      }
      if constexpr (C::OUT_BOXES > 0) {
        // The sums go out by way of shared memory, and the next tile's begin meanwhile.
        constexpr int COLS = OUT == GRAD_FP32 ? 32 : 64;
        const uint32_t out = base + C::SMEM_OUT + (warp - EPI_WARP0) * (C::OUT_BOXES * C::OUT_BOX);
        const int row = n0 - (int)lane / 4;
#pragma unroll
        for (int g = 0; g < 128 / COLS; ++g) {
          const uint32_t box = out + g % C::OUT_BOXES * C::OUT_BOX;
          if (lane == 0) bulk_wait_read<C::OUT_BOXES - 1>();
          __syncwarp();
          fill_box<OUT>(box, sum, g, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row < args.N && k0 + g * COLS < args.K)
              tma_store_3d_hint(&tmD, box, k0 + g * COLS, row, (int)t.e, pol);
            bulk_commit();
          }
        }
        continue;
      }
      // A split tile: the parts go into shared memory, and each pair adds up a stripe of rows, in
      // the pairs' order.  (A pair that gave up has said so, and the sums mean nothing.)
      const uint32_t mine = base + (warp - EPI_WARP0) * (64 * 32 * 8) + lane * 8;
      if constexpr (C::SPLIT > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(mine + (16 * i + 4 * g + j) * 256),
                           "f"(sum[i][g][j].x), "f"(sum[i][g][j].y)
                           : "memory");
        cluster_sync();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (C::SPLIT > 1 && i * C::SPLIT / 4 != (int)part) continue;
        const int64_t at = ((int64_t)t.e * args.N + n0 + 8 * i) * args.K + k8;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if constexpr (C::SPLIT > 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2 v[C::SPLIT];
#pragma unroll
              for (int q = 0; q < C::SPLIT; ++q)
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                             : "=f"(v[q].x), "=f"(v[q].y)
                             : "r"(mapa_shared(mine + (16 * i + 4 * g + j) * 256, q * C::CG + rank))
                             : "memory");
#pragma unroll
              for (int q = 1; q < C::SPLIT; ++q) {
                v[0].x += v[q].x;
                v[0].y += v[q].y;
              }
              sum[i][g][j] = v[0];
            }
          }
          store_row<OUT>(args.dB, at + 32 * g, sum[i][g], n0 + 8 * i < args.N && k8 + 32 * g < args.K,
                         wide, lane, pol);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  // the pair's MMAs and remote arrivals are finished before either CTA frees TMEM or exits
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<C::CG>(tmem_base, TMEM_COLS);
  }
}

template <class C, int OUT>
cudaError_t launch(const WgradArgs& args, int num_sms, cudaStream_t stream) {
  static_assert(smem_bytes<C>() <= 227 * 1024, "shared memory per CTA");
  CUtensorMap tmC, tmA, tmD = {};
  // with no rows nothing is loaded; a map still needs a row
  const uint64_t rows = args.M_total > 0 ? (uint64_t)args.M_total : 1;
  const uint64_t c_dims[2] = {(uint64_t)args.N, rows}, a_dims[2] = {(uint64_t)args.K, rows};
  if (!encode_swizzled(&tmC, C::FP8 ? 1 : 2, args.M_total > 0 ? args.dC : args.dB, 2, c_dims, C::ROWS) ||
      !encode_swizzled(&tmA, C::FP8 ? 1 : 2, args.M_total > 0 ? args.A : args.dB, 2, a_dims, C::ROWS))
    return cudaErrorInvalidValue;
  const uint64_t d_dims[3] = {(uint64_t)args.K, (uint64_t)args.N, (uint64_t)args.E};
  if (C::OUT_BOXES > 0 && !encode_swizzled(&tmD, OUT == GRAD_FP32 ? 4 : 2, args.dB, 3, d_dims, 32))
    return cudaErrorInvalidValue;
  CUtensorMap tmSC = {}, tmSA = {};
  if constexpr (C::FP8) {
    const uint64_t blocks = args.M_total / 128 + args.E;
    const bool any = args.M_total > 0;
    if (!encode_rows_f32(&tmSC, any ? args.dc_scales : args.dB, args.N, any ? blocks : 1, 128) ||
        !encode_rows_f32(&tmSA, any ? args.a_scales : args.dB, args.K, any ? blocks : 1, BN))
      return cudaErrorInvalidValue;
  }
  const cudaError_t e = allow_smem<wgrad_kernel<C, OUT>>(smem_bytes<C>());
  if (e != cudaSuccess) return e;
  const Shape shape = {(uint32_t)args.E, (uint32_t)((args.N + C::BM - 1) / C::BM),
                       (uint32_t)((args.K + BN - 1) / BN)};
  const int64_t tiles = (int64_t)shape.experts * shape.nt * shape.kt;
  const int64_t units = num_sms / C::CG;
  return launch_persistent(wgrad_kernel<C, OUT>, C::SPLIT > 1 || tiles < units ? tiles : units,
                           C::CG * C::SPLIT, THREADS, smem_bytes<C>(), stream, tmC, tmA, tmSC, tmSA, tmD,
                           args, shape);
}

template <class C>
int64_t at_once() {
  return clusters_at_once<wgrad_kernel<C, GRAD_FP32>>(C::CG * C::SPLIT, THREADS, smem_bytes<C>());
}

template <class C>
cudaError_t by_type(const WgradArgs& a, int num_sms, cudaStream_t stream) {
  switch (a.out_type) {
    case GRAD_BF16: return launch<C, GRAD_BF16>(a, num_sms, stream);
    case GRAD_FP16: return launch<C, GRAD_FP16>(a, num_sms, stream);
    default: return launch<C, GRAD_FP32>(a, num_sms, stream);
  }
}

using Split8 = Cfg<true, 128, 4, false, 4>;
using Split16 = Cfg<false, 128, 3, false, 4>;

}  // namespace wg

WgradPlan plan_wgrad(const WgradArgs& a, int num_sms, int64_t clusters) {
  // Few tiles and many rows: four pairs share a tile's rows (512 x 512: 8192 rows 54 -> 21 us; 304 x 416:
  // 1000 rows 12.6 -> 11.0, 3 groups of 900 12.4 -> 11.6, of 600 10.9 -> 11.5).
  const int64_t tiles = (int64_t)a.E * ((a.N + 255) / 256) * ((a.K + 255) / 256);
  if (a.M_total >= (int64_t)768 * a.E) {
    if (clusters < 0) clusters = a.fp8 ? wg::at_once<wg::Split8>() : wg::at_once<wg::Split16>();
    if (tiles <= clusters) return WgradPlan{128, 4, false};
  }
  // The gradients go out through shared memory and TMA, so that the epilogue takes up the next tile's
  // sums at once, or straight from the threads, in whole lines.  Which is faster was measured (32
  // experts of 2048 x 7168, us straight and by TMA):
  //   fp32 added to: straight, as the sums wait for what is added anyway and the stores then come
  //     evenly (8 bits, 256 rows each 627 and 765; 16 bits, 384 rows 643 and 730)
  //   fp32, short groups: straight, as the stores are what bounds it and mix worse with the operands'
  //     loads the further those run ahead (256 rows: 311 and 337, 8 bits 322 and 334); long groups or
  //     few tiles: TMA (512 rows 486 and 452, 8 bits 506 and 475; 8 experts of 2048 x 1024, 40 rows
  //     each, in 8 bits 18.0 and 16.0, 20 rows to bf16 12.6 and 11.5)
  //   16 bits out, half the bytes: TMA in 8 bits (256 rows 235 and 203) and where it is added to (464
  //     and 366), else straight (512 rows 380 and 391)
  const int64_t rounds = (tiles * 2 + num_sms - 1) / num_sms;
  const bool wide = a.out_type == GRAD_FP32;
  const bool long_groups = a.M_total >= (int64_t)384 * a.E;
  if (a.fp8) return WgradPlan{128, 1, !wide || (!a.add && (rounds <= 4 || long_groups))};
  return WgradPlan{long_groups ? 128 : 64, 1, a.add ? !wide : rounds <= 4 || (wide && long_groups)};
}

cudaError_t launch_wgrad(const WgradArgs& a, int num_sms, cudaStream_t stream) {
  const WgradPlan p = plan_wgrad(a, num_sms, -1);
  if (a.fp8) {
    if (p.split > 1) return wg::by_type<wg::Split8>(a, num_sms, stream);
    return p.staged ? wg::by_type<wg::Cfg<true, 128, 4, true>>(a, num_sms, stream)
                    : wg::launch<wg::Cfg<true, 128, 4, false>, GRAD_FP32>(a, num_sms, stream);
  }
  if (p.split > 1) return wg::by_type<wg::Split16>(a, num_sms, stream);
  if (p.rows == 128)
    return p.staged ? wg::by_type<wg::Cfg<false, 128, 3, true>>(a, num_sms, stream)
                    : wg::by_type<wg::Cfg<false, 128, 3, false>>(a, num_sms, stream);
  return p.staged ? wg::by_type<wg::Cfg<false, 64, 4, true>>(a, num_sms, stream)
                  : wg::by_type<wg::Cfg<false, 64, 4, false>>(a, num_sms, stream);
}

}  // namespace bsfp8
