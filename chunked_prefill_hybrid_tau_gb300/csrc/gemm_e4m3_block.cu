// Packed-token projections with block-scaled E4M3 operands (kind::f8f6f4):
//   C = epilogue(P),
//   P[m][n] = sum_b sa[m][b] sb[n / 128][b] sum_{k in block b} A[m][k] B[n][k]
// with A [M][K] token codes (one fp32 scale per row and 128 columns of K)
// and B [N][K] weight codes (one per 128 x 128 block), codes and scales as
// hb_quantize_e4m3_block writes them.
//
// The scales change along K, so the tensor cores cannot carry the sum over
// the blocks (the hardware's own block scales are powers of two per 32
// elements; these are any fp32 number per 128).  Each 128-wide K block is one
// accumulation in tensor memory; epilogue warps read it back and add it,
// scaled, to fp32 sums in registers:
//   acc = fma(part, fl(sa sb), acc), block by block in K order.
// Every kernel here adds the blocks of an output in this one order with
// these roundings, so a token's result does not depend on which kernel or
// tile its batch selected.
#include <cuda_bf16.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace {

using namespace dev;

constexpr int BM = 128;
constexpr int BK = 128;

struct Params {
  int M, N, K;
  int lda;
  void* C;
  const void* R;
  int ldc;       // row stride of C and R (elements)
  int out_cols;  // valid output columns (N, or N/2 for SWIGLU)
  const float* sa;
  const float* sb;
  int f_blocks;  // SWIGLU: rows of sb that belong to the gate
  int kblocks;
  int* status;
  bool preload;  // B was complete before the kernel ahead of this one: its first boxes do not wait for that kernel
  int rows;      // skinny kernel: weight rows of a tile
  int groups;    // skinny kernel: groups of NT tokens
  int stages;    // skinny kernel: ring depth
};

// silu(g) = g / (1 + e^-g), the arithmetic of the per-row scaled projections.
__device__ __forceinline__ float silu(float g) { return __fdividef(g, __fadd_rn(1.0f, __expf(-g))); }

// Byte offset of 16-byte chunk c (0..7) of row r in a slab of 128 rows x 128
// bytes with the 128-byte swizzle (the TMA box layout).
__device__ __forceinline__ uint32_t slab_off(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
constexpr int kSlabBytes = 128 * 128;

// Row of sb that scales B row n.  SWIGLU: B holds gate and up rows
// interleaved in blocks of 64, sb the gate's block scales, then the up's.
template <bool SWIGLU>
__device__ __forceinline__ int scale_row(const Params& p, int n) {
  if constexpr (SWIGLU) {
    const int f = (n >> 7) * 64 + (n & 63);
    return (f >> 7) + ((n & 64) ? p.f_blocks : 0);
  }
  return n >> 7;
}

__device__ __forceinline__ void tmem_ld_cols(uint32_t at, uint32_t (&r)[8]) { tmem_ld_32x32b_x8(at, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t at, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(at, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t at, uint32_t (&r)[32]) { tmem_ld_32x32b_x32(at, r); }

// ================================================================ wide tiles
// 128 x BN output tiles (PAIR: 256 x BN on a cluster of two CTAs with
// tcgen05 cta_group::2, each CTA holding its 128 rows of A and half of the B
// rows), persistent, M fastest so that the CTAs sharing a weight tile run
// together.
//   warps 0-7 : promotion and epilogue.  Warp w reads TMEM lanes 32 (w % 4)..
//               (its output rows) and column half w / 4, so a thread holds
//               BN / 2 fp32 sums of one row and scales a K block with one
//               factor (SWIGLU: one for its gate, one for its up columns);
//   warp 8    : TMA producer (128-byte swizzled boxes of one K block);
//   warps 9-10: MMA issuers.  TMEM holds four buffers of 128 columns; a K block
//               is BN / 128 of them, each with its own pair of barriers: at BN
//               = 256 every column half is refilled while the other is read.
//               The two warps take the column halves (BN 128: every second K
//               block): what one thread needs for its tries, MMAs and commits
//               is longer than the MMAs themselves;
//   warp 11   : fills the table of scales.
// The sums leave through shared memory staged apart from the ring and TMA
// stores, so the next tile's loads and MMAs go on meanwhile.
//
// A K block of a 256 x 256 pair tile is 512 clocks of MMAs; all of its 128 x 256
// partial sums then cross from TMEM to registers (256 clocks at 4 bytes a lane
// and clock) while the other half's MMAs update TMEM.  Measured: 750 clocks
// (394 ns).  4096 x 9216 x 7168: 191 us, 2.84 PFLOP/s, 145 at twice the measured
// bf16 rate; 512 x 28672 x 4096 (SWIGLU): 52 us, 2.31 PFLOP/s; both in a
// replayed graph.  Called one after the other for long, under the card's power
// limit: 212 and 56 us, 2.55 and 2.14 PFLOP/s.  (Without the
// epilogue 2% less, without A's loads 4%; the per-row scaled projection, the
// same MMAs without these sums: 156 and 41 us.)  Tried and
// slower: twice the promotion warps with half the sums each (255 against 225
// us, their waits and table reads double), packed fp32 FMAs, one issuing warp
// (207), 128-column tiles throughout (222).
constexpr int kTabK = 8;  // K blocks per fill of the scale table
constexpr int kBufs = 4;  // TMEM buffers of kSub columns
constexpr int kSub = 128;
template <int BN, bool PAIR>
struct Cfg {
  static constexpr int NSUB = BN / kSub;                            // buffers of a K block
  static constexpr int NB = kBufs / NSUB;                           // K blocks in TMEM
  static constexpr int SUB_BYTES = (PAIR ? kSub / 2 : kSub) * 128;  // B rows of one buffer (this CTA's)
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = NSUB * SUB_BYTES;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGING = BM * BN * 2;
  static constexpr int TABLE = kTabK * (BM + 4) * 4;  // one side: scales of the rows, then of up to 4 weight blocks
  static constexpr int AVAIL = 232448 - 1024 - 512 - STAGING - 2 * TABLE;
  static constexpr int STAGES = AVAIL / STAGE_BYTES < 8 ? AVAIL / STAGE_BYTES : 8;
  static constexpr int SMEM = STAGES * STAGE_BYTES + STAGING + 2 * TABLE + 512 + 1024;
  static constexpr int CH = BN / 64;  // 32-column chunks of a thread
  static_assert(BN == 128 || BN == 256, "BN");
  static_assert(STAGE_BYTES % 1024 == 0 && STAGING % 1024 == 0 && TABLE % 16 == 0, "alignment");
  static_assert(STAGES >= 3, "ring depth");
};
// 168 registers a thread at launch.  A promotion thread of a 256-column tile
// holds 128 sums and two sets of 16 columns on their way from TMEM; it gets
// 216 registers, the other warpgroup keeps 72 (4096 x 9216 x 7168: 201 us;
// 219 with 168 for all, where the next 16 columns cannot be under way).
constexpr int kWideThreads = 384;
constexpr int kIssueRegs = 72, kPromoteRegs = 216;
static_assert(128 * kIssueRegs + 256 * kPromoteRegs <= 168 * kWideThreads, "register split");

template <int BN, int EPI, bool PAIR>
__device__ __forceinline__ void wide_body(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC,
                                          const CUtensorMap& tmR, const Params& p) {
  using C = Cfg<BN, PAIR>;
  constexpr bool SWIGLU = EPI == HB_EPI_SWIGLU;
  constexpr int CH = C::CH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + C::STAGES * C::STAGE_BYTES;
  float* table = reinterpret_cast<float*>(staging + C::STAGING);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + C::STAGING + 2 * C::TABLE);  // PAIR: the even CTA's are used
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + kBufs;  // PAIR: the even CTA's are used
  uint64_t* tab_full = acc_empty + kBufs;
  uint64_t* tab_empty = tab_full + 2;
  uint64_t* drain = tab_empty + 2;
  uint64_t* res_bar = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int m_tiles = (p.M + BM - 1) / BM;
  const int um = PAIR ? (m_tiles + 1) / 2 : m_tiles;  // row tiles of a unit
  const int n_tiles = (p.N + BN - 1) / BN;
  const int units = um * n_tiles;
  const int first = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int stride = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
  const int kblocks = p.kblocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::NSUB);
    }
    for (int a = 0; a < kBufs; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], (PAIR ? 16 : 8) / C::NSUB);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tab_full[b], 32);
      mbar_init(&tab_empty[b], 8);
    }
    mbar_init(drain, 2);
    mbar_init(res_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 9) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full0 = PAIR ? cluster_addr(full, 0) : 0u;

  // (each setmaxnreg inside its role's own branch: the compiler allocates for
  // the smaller count where the two could meet)
  if (warp >= 8) {
    if constexpr (BN == 256) regs_dec<kIssueRegs>();
    if (warp == 8) {
      // ---------------------------------------------------------- TMA producer
      // The whole warp walks the loops and one elected lane issues (see the MMA
      // issuer): a single-lane loop needs twice the time per K block.
      const uint64_t wpol = um <= 4 ? policy_evict_first() : policy_evict_normal();
      const uint32_t empty_at = smem_u32(empty);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint32_t pending = 0, armed_parity = 0;
      auto load_a = [&](int s, int kb, int m0) {
        uint8_t* dst = smem + s * C::STAGE_BYTES;
        if constexpr (PAIR)
          tma_load_2d_pair(dst, &tmA, full0 + s * 8, kb * BK, m0);
        else
          tma_load_2d(dst, &tmA, &full[s], kb * BK, m0);
      };
      auto load_b = [&](int s, int kb, int n0) {
        uint8_t* dst = smem + s * C::STAGE_BYTES + C::A_BYTES;
#pragma unroll
        for (int i = 0; i < C::NSUB; ++i) {
          if constexpr (PAIR)
            tma_load_2d_pair_hint(dst + i * C::SUB_BYTES, &tmB, full0 + s * 8, kb * BK, n0 + i * kSub, wpol);
          else
            tma_load_2d_hint(dst + i * C::SUB_BYTES, &tmB, &full[s], kb * BK, n0 + i * kSub, wpol);
        }
      };
      auto arm = [&](int s) {
        if (leader) mbar_arrive_expect_tx(&full[s], (PAIR ? 2 : 1) * C::STAGE_BYTES);  // both CTAs' boxes
      };
      // weights that do not come from the kernel ahead: their first ring fill
      // is issued before waiting for it
      int pre = 0;
      if (p.preload && first < units) {
        const int n0 = (first / um) * BN + static_cast<int>(rank) * (kSub / 2);
        pre = kblocks < C::STAGES ? kblocks : C::STAGES;
        if (elect_one()) {
          for (int i = 0; i < pre; ++i) {
            arm(i);
            load_b(i, i, n0);
          }
        }
        __syncwarp();
      }
      griddep_wait();
      for (int u = first; u < units && ok; u += stride) {
        const int mt = PAIR ? 2 * (u % um) + static_cast<int>(rank) : u % um;
        const int n0 = (u / um) * BN + static_cast<int>(rank) * (kSub / 2);
#pragma unroll 1
        for (int kb = 0; kb < kblocks; ++kb) {
          pending |= 1u << stage;
          if (u == first && kb < pre) {
            if (elect_one()) load_a(stage, kb, mt * BM);
          } else {
            ok = __all_sync(0xffffffffu, mbar_wait_at(empty_at + stage * 8, phase ^ 1u, abort_flag, p.status));
            if (!ok) break;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            if (elect_one()) {
              arm(stage);
              load_a(stage, kb, mt * BM);
              load_b(stage, kb, n0);
            }
          }
          __syncwarp();
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (PAIR && *abort_flag) raise_peer_abort(abort_flag, rank);
      if (!ok) {
        // let copies already in flight land before the CTA leaves (one CTA:
        // their own barrier; a pair: the stage is released once consumed)
        for (int s = 0; s < C::STAGES; ++s)
          if (pending & (1u << s)) mbar_drain(PAIR ? &empty[s] : &full[s], (armed_parity >> s) & 1u);
      }
    } else if (warp == 9 || warp == 10) {
      // ---------------------------------------------------------- MMA issuers
      griddep_wait();
      if (leader) {
        // the whole warp walks the loop and one elected lane issues: inside a
        // single-lane branch every descriptor would be moved to a uniform
        // register anew
        constexpr uint32_t kIdesc = idesc_e4m3_f32(PAIR ? 2 * BM : BM, kSub);
        const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));
        const uint32_t full_at = smem_u32(full), acc_empty_at = smem_u32(acc_empty);
        const int me = warp - 9;
        // the K blocks (BN 128: every second one; their count runs over the
        // tiles) and the column half that are this warp's
        constexpr int STEP = C::NSUB == 2 ? 1 : 2;
        const int sub = C::NSUB == 2 ? me : 0;
        const uint32_t b_off = static_cast<uint32_t>((C::A_BYTES + sub * C::SUB_BYTES) >> 4);
        int stage = C::NSUB == 2 ? 0 : me, slot = stage;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        const int mine = (units - first + stride - 1) / stride;  // tiles of this CTA
        const long long blocks = mine > 0 ? static_cast<long long>(mine) * kblocks : 0;
#pragma unroll 1
        for (long long kb = C::NSUB == 2 ? 0 : me; kb < blocks; kb += STEP) {
          const int buf = sub * C::NB + slot;
          const uint32_t buf_at = acc_empty_at + buf * 8, data_at = full_at + stage * 8;
          if constexpr (C::NSUB == 2) {
            // this warp has waited for every phase of both barriers, so both
            // are tried before either vote: one after the other, tries and
            // votes took as long as the MMAs
            const bool has_buf = mbar_try_wait_at(buf_at, bphase ^ 1u);
            const bool has_data = mbar_try_wait_at(data_at, phase);
            ok = __all_sync(0xffffffffu, has_buf && has_data) ||
                 __all_sync(0xffffffffu, mbar_wait_at(buf_at, bphase ^ 1u, abort_flag, p.status) &&
                                             mbar_wait_at(data_at, phase, abort_flag, p.status));
          } else {
            // The buffer first, and the operands only once it is known to be
            // free: the other warp had this stage before, and a wait by parity
            // also passes while that earlier phase is still open.  Tried
            // together, the operands' barrier can be looked at while the
            // buffer's try is pending; taken for complete one phase early, it
            // let a block's MMAs run on half a stage and free it twice.  A
            // released buffer means that block kb - NB has been summed, so
            // every block up to it has left the ring, kb - STAGES among them.
            static_assert(C::STAGES > C::NB, "a stage's earlier phase is over when its buffer is free");
            ok = __all_sync(0xffffffffu, mbar_wait_at(buf_at, bphase ^ 1u, abort_flag, p.status));
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_at(data_at, phase, abort_flag, p.status));
          }
          if (!ok) break;
          tc_fence_after();
          // the start address is the low 14 bits of a descriptor, in 16-byte
          // units, and shared memory ends below 2^18 bytes: it cannot carry
          const uint64_t a_desc = desc0 + static_cast<uint32_t>(stage * (C::STAGE_BYTES >> 4));
          const uint64_t b_desc = a_desc + b_off;
          const uint32_t d_tmem = tmem_base + buf * kSub;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (PAIR)
                mma_e4m3_pair(d_tmem, a_desc + 2 * k, b_desc + 2 * k, kIdesc, k != 0);
              else
                mma_e4m3(d_tmem, a_desc + 2 * k, b_desc + 2 * k, kIdesc, k != 0);
            }
            // the buffer last: its arrival is the one that the sums, and so the
            // end of a CTA, wait for
            if constexpr (PAIR) {
              mma_commit_pair(&empty[stage], 3);
              mma_commit_pair(&acc_full[buf], 3);
            } else {
              mma_commit(&empty[stage]);
              mma_commit(&acc_full[buf]);
            }
          }
          __syncwarp();
          stage += STEP;
          if (stage >= C::STAGES) {
            stage -= C::STAGES;
            phase ^= 1u;
          }
          slot += STEP;
          if (slot >= C::NB) {
            slot -= C::NB;
            bphase ^= 1u;
          }
        }
        if (PAIR && *abort_flag) raise_peer_abort(abort_flag, rank);
        // no MMA may still read shared memory or write tensor memory when the CTAs leave
        if (elect_one()) {
          if constexpr (PAIR)
            mma_commit_pair(drain, 1);
          else
            mma_commit(drain);
        }
        __syncwarp();
        mbar_drain(drain, 0);
      }
    } else {
      // ---------------------------------------------------------- scale table
      // Scales of the tile's rows and weight blocks, kTabK K blocks at a time,
      // two fills ahead of the sums.  (Read by the promotion warps themselves,
      // each row of sa is a cache line of its own: 128 lines and the few spills
      // outgrew the L1 left beside the ring, and a K block took three times as
      // long.)
      griddep_wait();
      int fill = 0;
      bool ok = true;
      for (int u = first; u < units; u += stride) {
        const int mt = PAIR ? 2 * (u % um) + static_cast<int>(rank) : u % um;
        const int n0 = (u / um) * BN;
        const float* pa[4];
        bool in_m[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = mt * BM + q * 32 + lane;
          in_m[q] = row < p.M;
          pa[q] = p.sa + static_cast<size_t>(in_m[q] ? row : 0) * kblocks;
        }
        // weight block j: buffer j / 2's gate (or only) block, and its up block
        const int j = lane & 3;
        const int n = n0 + (BN == 256 ? (j >> 1) * kSub : 0) + (SWIGLU ? (j & 1) * 64 : 0);
        const float* ps =
            p.sb + static_cast<size_t>(scale_row<SWIGLU>(p, n < p.N ? n : p.N - 1)) * kblocks + (lane >> 2);
        for (int kb0 = 0; kb0 < kblocks; kb0 += kTabK, ++fill) {
          float va[4][kTabK];
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < kTabK; ++i) va[q][i] = kb0 + i < kblocks && in_m[q] ? ld_f32(pa[q] + kb0 + i) : 0.f;
          const float vs = kb0 + (lane >> 2) < kblocks ? ld_f32(ps + kb0) : 0.f;
          const int b = fill & 1;
          if (ok) ok = mbar_wait(&tab_empty[b], ((fill >> 1) & 1) ^ 1u, abort_flag, p.status);
          float* tab = table + b * (C::TABLE / 4);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < kTabK; ++i) tab[i * BM + q * 32 + lane] = va[q][i];
          tab[kTabK * BM + lane] = vs;
          mbar_arrive(&tab_full[b]);
        }
      }
    }
  } else {
    // ---------------------------------------------------------- promotion and epilogue
    if constexpr (BN == 256) regs_inc<kPromoteRegs>();
    griddep_wait();
    const int quarter = warp & 3, half = warp >> 2;
    const bool boss = threadIdx.x == 0;
    const int rloc = quarter * 32 + lane;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    // first column of chunk c of this half.  SWIGLU, BN 128: 32 gate columns
    // and the 32 up columns that go with them.
    auto chunk_col = [&](int c) {
      if (SWIGLU && BN == 128) return half * 32 + c * 64;
      return half * (BN / 2) + c * 32;
    };
    // column half w / 4: at BN 256 a buffer of its own
    const int sub = BN == 256 ? half : 0;
    // addresses as one register and constants: at BN = 256 the sums leave few
    const uint32_t bars = smem_u32(full);
    const uint32_t acc_full_at = bars + (2 * C::STAGES + sub * C::NB) * 8, acc_empty_at = acc_full_at + kBufs * 8;
    const uint32_t acc_empty_peer = PAIR ? cluster_addr_at(acc_empty_at, 0) : 0u;
    const uint32_t tab_full_at = bars + (2 * C::STAGES + 2 * kBufs) * 8, tab_empty_at = tab_full_at + 16;
    const uint32_t sa_at = bars - 2 * C::TABLE + rloc * 4;
    const uint32_t sb_at = bars - 2 * C::TABLE + (kTabK * BM + half * 2) * 4;
    int fill = 0, slot = 0;
    uint32_t bphase = 0, rphase = 0;
    bool ok = true;
    bool res_pending = false;  // boss: residual copies in flight
    for (int u = first; u < units; u += stride) {
      const int mt = PAIR ? 2 * (u % um) + static_cast<int>(rank) : u % um;
      const int n0 = (u / um) * BN;
      const bool live = mt < m_tiles;  // a pair's odd row tile may lie past M
      float acc[CH][32];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c][j] = 0.f;
      // The sums run over W columns at a time, the next W on their way from
      // TMEM meanwhile, across the border of two K blocks too.  A wait that
      // expired raises the abort flag, a thread whose wait has failed waits
      // for nothing any more (a tile more then costs its arithmetic, however
      // many K blocks are left), and the loop runs on over whatever TMEM
      // holds: no buffer is released any more, and nothing of the tile is
      // stored.  A tile is the work of all eight warps, whose waits need not
      // expire together (at BN 256 the halves have buffers of their own), so
      // the store asks the flag, which every warp has had its chance to raise
      // before the barrier ahead of it.
      constexpr int W = BN == 256 && EPI != HB_EPI_F32 ? 32 : 16;  // (F32 at 32 spilled: 246 us against 229)
      constexpr int NC = CH * 32 / W;
      uint32_t r[2][W];
      const uint32_t t_cols = t_lane + sub * C::NB * kSub - sub * kSub;
      auto step_col = [&](int c) { return chunk_col(c * W / 32) + c * W % 32; };
      // waits for the next K block in TMEM and starts its first columns;
      // there: an earlier try has found it complete
      auto next_block = [&](bool there) {
        if (!__all_sync(0xffffffffu, there)) {
          if (ok) ok = mbar_wait_at(acc_full_at + slot * 8, bphase, abort_flag, p.status);
          __syncwarp();
        }
        tc_fence_after();
        tmem_ld_cols(t_cols + slot * kSub + step_col(0), r[0]);
      };
      next_block(false);
#pragma unroll 1
      for (int kb0 = 0; kb0 < kblocks; kb0 += kTabK, ++fill) {
        const int side = fill & 1;
        const int nk = kblocks - kb0 < kTabK ? kblocks - kb0 : kTabK;
        if (ok) ok = mbar_wait_at(tab_full_at + side * 8, (fill >> 1) & 1, abort_flag, p.status);
        __syncwarp();
        uint32_t sa_next = sa_at + side * C::TABLE, sb_next = sb_at + side * C::TABLE;
        if constexpr (EPI == HB_EPI_RESIDUAL) {
          // the residual tile into the staging slabs, once the previous
          // tile's stores have left them (in the second round: long done)
          if (boss && live && ok && kb0 == (kblocks > kTabK ? kTabK : 0)) {
            bulk_wait_group_read<0>();
            int slabs = (p.N - n0 + 63) / 64;
            if (slabs > BN / 64) slabs = BN / 64;
            mbar_arrive_expect_tx(res_bar, slabs * kSlabBytes);
#pragma unroll 1
            for (int s = 0; s < slabs; ++s)
              tma_load_2d(staging + s * kSlabBytes, &tmR, res_bar, n0 + s * 64, mt * BM);
            res_pending = true;
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int i = 0; i < nk; ++i) {
          const float sa = lds_f32(sa_next);
          const float2 sb = lds_f32x2(sb_next);
          sa_next += BM * 4;
          sb_next += 16;
          const float f0 = __fmul_rn(sa, sb.x), f1 = SWIGLU ? __fmul_rn(sa, sb.y) : f0;
          const bool more = kb0 + i + 1 < kblocks, wrap = slot + 1 == C::NB;
          const int next_slot = !more ? slot : wrap ? 0 : slot + 1;
          const uint32_t next_phase = more && wrap ? bphase ^ 1u : bphase;
          bool there = false;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            tmem_ld_wait();
            // Late enough to find it, early enough that its latency passes
            // under the sums.  Past the tile's last block there is nothing to
            // find, and a try would hold the thread in vain: it takes the
            // present block, which is complete.
            if (c == NC - 2) there = mbar_try_wait_at(acc_full_at + next_slot * 8, next_phase);
            if (c < NC - 1) tmem_ld_cols(t_cols + slot * kSub + step_col(c + 1), r[(c + 1) & 1]);
            if (c == NC - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0 && ok) {
                if constexpr (PAIR)
                  mbar_arrive_cluster_relaxed(acc_empty_peer + slot * 8);
                else
                  mbar_arrive_at(acc_empty_at + slot * 8);
              }
              if (++slot == C::NB) {
                slot = 0;
                bphase ^= 1u;
              }
              if (more) next_block(there);
            }
            // scalar FMAs: the packed fma.rn.f32x2 needs register pairs that
            // the TMEM load does not give without moves (620 against 370
            // clocks per 256-column block, measured)
            const float f = c < NC / 2 ? f0 : f1;
#pragma unroll
            for (int j = 0; j < W; ++j) {
              float& a = acc[c * W / 32][c * W % 32 + j];
              a = __fmaf_rn(__uint_as_float(r[c & 1][j]), f, a);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_at(tab_empty_at + side * 8);
      }
      ok = __all_sync(0xffffffffu, ok);
      // ---- the tile's sums are complete
      if (!live) continue;  // the same for every thread of the CTA
      if constexpr (EPI == HB_EPI_RESIDUAL) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(res_bar, rphase, abort_flag, p.status));
        if (ok) {
          rphase ^= 1u;
          res_pending = false;
        }
      } else {
        if (boss) bulk_wait_group_read<0>();
        __syncwarp();
        named_barrier_sync(1, 256);
      }
      if constexpr (EPI == HB_EPI_F32) {
        constexpr int ROUNDS = 2, PER = CH / 2;  // chunks of a half and round; one 32-column slab each
#pragma unroll
        for (int rd = 0; rd < ROUNDS; ++rd) {
          if (rd > 0) {
            if (boss) bulk_wait_group_read<0>();
            __syncwarp();
            named_barrier_sync(1, 256);
          }
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            uint8_t* slab = staging + (half * PER + i) * kSlabBytes;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float* v = &acc[rd * PER + i][4 * q];
              *reinterpret_cast<float4*>(slab + slab_off(rloc, q)) = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
          fence_proxy_async_smem();
          named_barrier_sync(2, 256);
          if (boss && all_waits_held(ok, abort_flag)) {
            for (int h = 0; h < 2; ++h)
              for (int i = 0; i < PER; ++i) {
                const int x = n0 + h * (BN / 2) + (rd * PER + i) * 32;
                if (x < p.out_cols) tma_store_2d(&tmC, staging + (h * PER + i) * kSlabBytes, x, mt * BM);
              }
            bulk_commit_group();
          }
        }
      } else {
        if constexpr (SWIGLU) {
          // BN 256: chunks 0, 1 gate and 2, 3 up of one 64-column output
          // slab per half; BN 128: one chunk of each, half a slab per half
          constexpr int G = CH / 2;
#pragma unroll
          for (int i = 0; i < G; ++i) {
            uint8_t* slab = staging + (BN == 256 ? half : 0) * kSlabBytes;
            const int c0 = (BN == 256 ? i : half) * 4;  // first 16-byte piece
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int e = 8 * q + 2 * j;
                w[j] = pack_bf16x2(__fmul_rn(silu(acc[i][e]), acc[G + i][e]),
                                   __fmul_rn(silu(acc[i][e + 1]), acc[G + i][e + 1]));
              }
              *reinterpret_cast<uint4*>(slab + slab_off(rloc, c0 + q)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int col = half * (BN / 2) + c * 32;
            uint8_t* slab = staging + (col >> 6) * kSlabBytes;
            const int c0 = (col & 32) >> 3;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4* dst = reinterpret_cast<uint4*>(slab + slab_off(rloc, c0 + q));
              uint32_t w[4];
              if constexpr (EPI == HB_EPI_RESIDUAL) {
                const uint4 rv = *dst;
                const uint32_t rr[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 f = unpack_bf16x2(rr[j]);
                  w[j] = pack_bf16x2(__fadd_rn(f.x, acc[c][8 * q + 2 * j]), __fadd_rn(f.y, acc[c][8 * q + 2 * j + 1]));
                }
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(acc[c][8 * q + 2 * j], acc[c][8 * q + 2 * j + 1]);
              }
              *dst = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        fence_proxy_async_smem();
        named_barrier_sync(2, 256);
        if (boss && all_waits_held(ok, abort_flag)) {
          constexpr int SLABS = SWIGLU ? BN / 128 : BN / 64;
          const int x0 = SWIGLU ? n0 / 2 : n0;
          for (int s = 0; s < SLABS; ++s)
            if (x0 + s * 64 < p.out_cols) tma_store_2d(&tmC, staging + s * kSlabBytes, x0 + s * 64, mt * BM);
          bulk_commit_group();
        }
      }
    }
    if (res_pending) mbar_drain(res_bar, rphase);
    if (boss) bulk_wait_group<0>();  // the TMA stores have left shared memory and are performed
    if (PAIR && lane == 0 && *abort_flag) raise_peer_abort(abort_flag, rank);
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

template <int BN, int EPI>
__global__ void __launch_bounds__(kWideThreads, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR, Params p) {
  wide_body<BN, EPI, false>(tmA, tmB, tmC, tmR, p);
}

template <int BN, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    block_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR, Params p) {
  wide_body<BN, EPI, true>(tmA, tmB, tmC, tmR, p);
}

// ================================================================ few tokens
// The weights are the bound, so the operands change places: a tile is p.rows
// weight rows (TMEM lanes) x NT tokens (columns), and the rows per tile are
// chosen so that the tiles fill the SMs; more than NT tokens make groups, the
// tiles of one weight box side by side.  The MMA has M = 64, or 128 above 64
// rows: lanes past p.rows multiply whatever follows in shared memory and are
// not read.
//
// With one issuing warp, M = 128 and one promotion warp a lane, a K block cost
// the steps in turn of one warp (wait, four MMAs, commit; 290 clocks).  So K
// blocks go through the ring in pairs, one for each of two issuing warps, and
// through TMEM in groups of four, and the sums of a lane are shared by two
// warps.  What is left is about 107 clocks and 2.2 for each 128-byte row of
// weights and tokens (48, 64 and 96 rows: 213, 240 and 320 clocks): an SM takes
// in 64 bytes a clock from L2, the tokens' rows included.  Four issuing warps are
// no faster.  Calls in a replayed graph, and in brackets with the weights'
// first boxes fetched ahead of the wait, as in a layer: 32 x 4096 x 14336 18.7
// us (17.3; 8.8 at the copy rate), 1 x 6144 x 4096 7.1 (7.2), 1 x 28672 x 4096
// (SWIGLU) 20.8, 5.7 TB/s (19.3), 32 x 128256 x 4096 (F32) 75.9, 7.0 TB/s
// (74.4).
//   warps 0-7: promotion and epilogue, warp w for TMEM lanes 32 (w % 4).. (those
//              below p.rows) and half w / 4 of the tokens; all eight fill the
//              table of scale products;
//   warp 8   : TMA producer;
//   warps 9-10: MMA issuers, one K block of every stage each.
constexpr int kSkinnyThreads = 352;
constexpr int kGroup = 4;       // K blocks of one TMEM buffer
constexpr int kSkinnyTabK = 16; // K blocks per fill of the scale table

template <int NT>
struct CfgSkinny {
  static constexpr int NBUF = NT == 64 ? 2 : 4;
  static constexpr int TMEM_COLS = NBUF * kGroup * NT;
  static constexpr int TH = NT / 2;                 // tokens of a promotion thread
  static constexpr int LOADS = NT == 64 ? 2 : kGroup;  // K blocks read from TMEM at a time
  static constexpr int TAB = kSkinnyTabK * 2 * NT;  // floats of one buffer: [K block][weight block][token]
  static constexpr int MAX_STAGES = 16;
  static constexpr int BAR_BYTES = 512;
  static constexpr int XCH_BYTES = 64 * (NT + 1) * 4;  // SWIGLU: up sums for the gate's threads
  static constexpr int FIXED = 1024 + BM * 128 + 2 * TAB * 4 + BAR_BYTES + XCH_BYTES;
  static_assert(NT == 16 || NT == 32 || NT == 64, "NT");
};

template <int NT, int EPI>
__global__ void __launch_bounds__(kSkinnyThreads, 1)
    block_gemm_skinny_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                             Params p) {
  using C = CfgSkinny<NT>;
  constexpr bool SWIGLU = EPI == HB_EPI_SWIGLU;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int w_bytes = p.rows * 128, kb_bytes = w_bytes + NT * 128, stage_bytes = 2 * kb_bytes;
  // BM * 128 bytes past the ring: the last stage's MMAs read their unused lanes there
  float* table = reinterpret_cast<float*>(smem + p.stages * stage_bytes + BM * 128);
  float* xch = table + 2 * C::TAB;
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(xch) + C::XCH_BYTES);
  uint64_t* empty = full + C::MAX_STAGES;
  uint64_t* acc_full = empty + C::MAX_STAGES;
  uint64_t* acc_empty = acc_full + C::NBUF;
  uint64_t* drain = acc_empty + C::NBUF;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;
  const int kblocks = p.kblocks;
  const int pairs = (kblocks + 1) / 2;  // ring stages of a tile (past K the boxes are zeros)
  const int R = p.rows, G = R / 2;
  const int per_block = SWIGLU ? 64 / G : 1;  // SWIGLU tiles of one 128-row gate/up block
  // the groups of one weight tile run side by side
  const int tiles = (SWIGLU ? (p.N / 128) * per_block : (p.N + R - 1) / R) * p.groups;
  const bool m64 = R <= 64;
  const int act_warps = m64 ? (R + 15) / 16 : (R + 31) / 32;
  const int ring = p.stages;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ring; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
    }
    for (int a = 0; a < C::NBUF; ++a) {
      mbar_init(&acc_full[a], 2);
      mbar_init(&acc_empty[a], 2 * act_warps);
    }
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 8) {
    // ---------------------------------------------------------- TMA producer
    const uint64_t wpol = policy_evict_first();  // a weight box is read once, or by its groups side by side
    const uint32_t empty_at = smem_u32(empty);
    auto load_w = [&](int s, int pr, int t) {
      const int wt = t / p.groups;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint8_t* dst = smem + s * stage_bytes + h * kb_bytes;
        const int k = (2 * pr + h) * BK;
        if constexpr (SWIGLU) {
          const int n = (wt / per_block) * 128 + (wt % per_block) * G;
          tma_load_2d_hint(dst, &tmB, &full[s], k, n, wpol);
          tma_load_2d_hint(dst + G * 128, &tmB, &full[s], k, n + 64, wpol);
        } else {
          tma_load_2d_hint(dst, &tmB, &full[s], k, wt * R, wpol);
        }
      }
    };
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    uint32_t pending = 0, armed_parity = 0;
    const int t0 = static_cast<int>(blockIdx.x);
    int pre = 0;
    if (p.preload && t0 < tiles) {
      pre = pairs < ring ? pairs : ring;
      if (elect_one()) {
        for (int i = 0; i < pre; ++i) {
          mbar_arrive_expect_tx(&full[i], stage_bytes);
          load_w(i, i, t0);
        }
      }
      __syncwarp();
    }
    griddep_wait();
    for (int t = t0; t < tiles && ok; t += gridDim.x) {
      const int m0 = t % p.groups * NT;
#pragma unroll 1
      for (int pr = 0; pr < pairs; ++pr) {
        const bool fresh = !(t == t0 && pr < pre);
        pending |= 1u << stage;
        if (fresh) {
          ok = __all_sync(0xffffffffu, mbar_wait_at(empty_at + stage * 8, phase ^ 1u, abort_flag, p.status));
          if (!ok) break;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        }
        if (elect_one()) {
          if (fresh) {
            mbar_arrive_expect_tx(&full[stage], stage_bytes);
            load_w(stage, pr, t);
          }
          uint8_t* dst = smem + stage * stage_bytes + w_bytes;
          tma_load_2d(dst, &tmA, &full[stage], 2 * pr * BK, m0);
          tma_load_2d(dst + kb_bytes, &tmA, &full[stage], (2 * pr + 1) * BK, m0);
        }
        __syncwarp();
        if (++stage == ring) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok)
      for (int s = 0; s < ring; ++s)
        if (pending & (1u << s)) mbar_drain(&full[s], (armed_parity >> s) & 1u);
  } else if (warp >= 9) {
    // ---------------------------------------------------------- MMA issuers
    griddep_wait();
    const uint32_t idesc = m64 ? idesc_e4m3_f32(64, NT) : idesc_e4m3_f32(BM, NT);
    // the two warps take one K block of every stage each
    const int me = warp - 9;
    const uint64_t desc0 = smem_desc_sw128(smem_u32(smem) + me * kb_bytes);
    const uint32_t tmem_me = tmem_base + me * NT;
    const uint32_t full_at = smem_u32(full), acc_empty_at = smem_u32(acc_empty);
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
#pragma unroll 1
      for (int pr = 0; pr < pairs; ++pr) {
        const int in_group = pr % (kGroup / 2);
        ok = mbar_wait_at(full_at + stage * 8, phase, abort_flag, p.status);
        if (in_group == 0) ok = ok && mbar_wait_at(acc_empty_at + buf * 8, bphase ^ 1u, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const bool last = in_group == kGroup / 2 - 1 || pr == pairs - 1;
        if (elect_one()) {
          const uint64_t w_desc = desc0 + static_cast<uint32_t>((stage * stage_bytes) >> 4);
          const uint64_t x_desc = w_desc + static_cast<uint32_t>(w_bytes >> 4);
          const uint32_t d = tmem_me + (buf * kGroup + in_group * 2) * NT;
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_e4m3(d, w_desc + 2 * k, x_desc + 2 * k, idesc, k != 0);
          mma_commit(&empty[stage]);
          if (last) mma_commit(&acc_full[buf]);
        }
        __syncwarp();
        if (++stage == ring) {
          stage = 0;
          phase ^= 1u;
        }
        if (last && ++buf == C::NBUF) {
          buf = 0;
          bphase ^= 1u;
        }
      }
    }
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mbar_drain(drain, 0);
  } else {
    // ---------------------------------------------------------- promotion and epilogue
    griddep_wait();
    constexpr int TH = C::TH;
    const int quarter = warp & 3, j0 = (warp >> 2) * TH;  // this warp's first token
    const bool active = quarter < act_warps;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + j0;
    // weight row within the tile (M = 64: rows 16 w.. in lanes 32 w..)
    const int e = m64 ? (lane < 16 ? quarter * 16 + lane : BM) : quarter * 32 + lane;
    // Scale products of K block kb0 + fi, fi = threadIdx.x % kSkinnyTabK:
    // thread's tokens fj, fj + 16, ...; the two weight blocks a tile can touch
    // (SWIGLU: the gate's and the up's).
    constexpr int PER = NT / 16;
    const int fi = threadIdx.x % kSkinnyTabK, fj = threadIdx.x / kSkinnyTabK;
    float pre_a[PER], pre_b[2];
    const float* sb_blk[2];
    int m0 = 0;  // the tile's first token
    auto fetch = [&](int kb0) {
      const bool in = kb0 + fi < kblocks;
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int j = m0 + fj + 16 * x;
        pre_a[x] = in && j < p.M ? ld_f32(p.sa + static_cast<size_t>(j) * kblocks + kb0 + fi) : 0.f;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) pre_b[b] = in ? ld_f32(sb_blk[b] + kb0 + fi) : 0.f;
    };
    auto put = [&](int side) {
#pragma unroll
      for (int x = 0; x < PER; ++x)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          table[side * C::TAB + (fi * 2 + b) * NT + fj + 16 * x] = __fmul_rn(pre_a[x], pre_b[b]);
    };
    const uint32_t table_at = smem_u32(table) + j0 * 4;
    const uint32_t acc_full_at = smem_u32(acc_full), acc_empty_at = smem_u32(acc_empty);
    int buf = 0;
    uint32_t bphase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int wt = t / p.groups;
      m0 = (t - wt * p.groups) * NT;
      int n;    // this thread's row of B
      bool n_ok;
      int blk;  // which of the tile's two weight blocks scales it
      if constexpr (SWIGLU) {
        const int base = (wt / per_block) * 128;
        n = base + (wt % per_block) * G + (e < G ? e : 64 + e - G);
        n_ok = e < R;
        blk = n_ok && e >= G ? 1 : 0;
        for (int b = 0; b < 2; ++b) sb_blk[b] = p.sb + static_cast<size_t>(scale_row<true>(p, base + 64 * b)) * kblocks;
      } else {
        n = wt * R + e;
        n_ok = e < R && n < p.N;
        const int b0 = wt * R / BK, b1 = (p.N - 1) / BK;
        blk = n_ok ? n / BK - b0 : 0;
        sb_blk[0] = p.sb + static_cast<size_t>(b0) * kblocks;
        sb_blk[1] = p.sb + static_cast<size_t>(b0 < b1 ? b0 + 1 : b1) * kblocks;
      }
      float acc[TH];
#pragma unroll
      for (int j = 0; j < TH; ++j) acc[j] = 0.f;
      fetch(0);
      // the residuals of this thread's outputs, read while the first boxes
      // arrive (each read behind the last output's store, which may alias it,
      // they cost 5 us for 64 tokens)
      [[maybe_unused]] uint32_t res[TH / 2];
      if constexpr (EPI == HB_EPI_RESIDUAL) {
        const auto* rp = static_cast<const uint16_t*>(p.R) + (n_ok ? n : 0);
        uint32_t v[TH];
#pragma unroll
        for (int j = 0; j < TH; ++j) {
          const int row = m0 + j0 + j < p.M ? m0 + j0 + j : p.M - 1;
          v[j] = rp[static_cast<size_t>(row) * p.ldc];
        }
#pragma unroll
        for (int j = 0; j < TH; j += 2) res[j / 2] = v[j] | (v[j + 1] << 16);
      }
      named_barrier_sync(1, 256);  // the previous tile's table reads are done
      put(0);
#pragma unroll 1
      for (int kb0 = 0; kb0 < kblocks; kb0 += kGroup) {
        const int ti = kb0 % kSkinnyTabK, side = (kb0 / kSkinnyTabK) & 1;
        if (ti == 0) {
          named_barrier_sync(1, 256);  // this side of the table is filled, the other one is read
          if (kb0 + kSkinnyTabK < kblocks) fetch(kb0 + kSkinnyTabK);
        }
        if (ti == kSkinnyTabK - kGroup && kb0 + kGroup < kblocks) put(side ^ 1);
        if (active) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait_at(acc_full_at + buf * 8, bphase, abort_flag, p.status));
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int g0 = 0; g0 < kGroup; g0 += C::LOADS) {
              uint32_t r[C::LOADS][TH];
#pragma unroll
              for (int g = 0; g < C::LOADS; ++g) tmem_ld_cols(t_lane + (buf * kGroup + g0 + g) * NT, r[g]);
              tmem_ld_wait();
              if (g0 + C::LOADS == kGroup) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(acc_empty_at + buf * 8);
              }
#pragma unroll
              for (int g = 0; g < C::LOADS; ++g) {
                if (kb0 + g0 + g >= kblocks) break;
                const uint32_t at = table_at + (side * C::TAB + ((ti + g0 + g) * 2 + blk) * NT) * 4;
#pragma unroll
                for (int j = 0; j < TH; j += 4) {
                  const float4 f = lds_f32x4(at + j * 4);
                  acc[j] = __fmaf_rn(__uint_as_float(r[g][j]), f.x, acc[j]);
                  acc[j + 1] = __fmaf_rn(__uint_as_float(r[g][j + 1]), f.y, acc[j + 1]);
                  acc[j + 2] = __fmaf_rn(__uint_as_float(r[g][j + 2]), f.z, acc[j + 2]);
                  acc[j + 3] = __fmaf_rn(__uint_as_float(r[g][j + 3]), f.w, acc[j + 3]);
                }
              }
            }
          }
        }
        if (++buf == C::NBUF) {
          buf = 0;
          bphase ^= 1u;
        }
      }
      // ---- the tile's sums are complete: token j of output column n
      if constexpr (SWIGLU) {
        if (active && e >= G && e < R) {
#pragma unroll
          for (int j = 0; j < TH; ++j) xch[(e - G) * (NT + 1) + j0 + j] = acc[j];
        }
        named_barrier_sync(1, 256);
        // the up sums are another warp's
        if (active && e < G && all_waits_held(ok, abort_flag)) {
          const int f = (wt / per_block) * 64 + (wt % per_block) * G + e;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.C) + f;
#pragma unroll
          for (int j = 0; j < TH; ++j)
            if (m0 + j0 + j < p.M)
              dst[static_cast<size_t>(m0 + j0 + j) * p.ldc] =
                  __float2bfloat16_rn(__fmul_rn(silu(acc[j]), xch[e * (NT + 1) + j0 + j]));
        }
      } else if (active && ok && n_ok) {
#pragma unroll
        for (int j = 0; j < TH; ++j) {
          if (m0 + j0 + j >= p.M) continue;
          const size_t at = static_cast<size_t>(m0 + j0 + j) * p.ldc + n;
          if constexpr (EPI == HB_EPI_F32) {
            static_cast<float*>(p.C)[at] = acc[j];
          } else if constexpr (EPI == HB_EPI_RESIDUAL) {
            const float2 pair = unpack_bf16x2(res[j / 2]);
            const float r = j & 1 ? pair.y : pair.x;
            static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(__fadd_rn(r, acc[j]));
          } else {
            static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(acc[j]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- launches
template <int BN, int EPI, bool PAIR>
hb_status launch_wide(const DeviceCtx& ctx, const void* A, const void* B, const Params& p, cudaStream_t stream) {
  using C = Cfg<BN, PAIR>;
  CUtensorMap tmA, tmB, tmC, tmR;
  hb_status st = encode_tmap_2d(&tmA, A, p.K, p.M, p.lda, BK, BM, true, 1);
  if (st != HB_OK) return st;
  st = encode_tmap_2d(&tmB, B, p.K, p.N, p.K, BK, PAIR ? kSub / 2 : kSub, true, 1);
  if (st != HB_OK) return st;
  constexpr int ESZ = EPI == HB_EPI_F32 ? 4 : 2;
  st = encode_tmap_2d(&tmC, p.C, p.out_cols, p.M, static_cast<uint64_t>(p.ldc) * ESZ, 128 / ESZ, BM, true, ESZ);
  if (st != HB_OK) return st;
  if (EPI == HB_EPI_RESIDUAL) {
    st = encode_tmap_2d(&tmR, p.R, p.out_cols, p.M, static_cast<uint64_t>(p.ldc) * 2, 64, BM, true, 2);
    if (st != HB_OK) return st;
  } else {
    tmR = tmC;
  }
  static std::atomic<bool> attr_set[kMaxDevices];
  const int m_tiles = (p.M + BM - 1) / BM, n_tiles = (p.N + BN - 1) / BN;
  if constexpr (PAIR) {
    st = smem_limit_once(attr_set, ctx.device, block_gemm_pair_kernel<BN, EPI>, C::SMEM,
                         "cudaFuncSetAttribute(block gemm pair)");
    if (st != HB_OK) return st;
    const int units = (m_tiles + 1) / 2 * n_tiles, pairs = ctx.num_sms / 2;
    return launch_pdl(block_gemm_pair_kernel<BN, EPI>, 2 * (units < pairs ? units : pairs), kWideThreads, C::SMEM,
                      stream, "block_gemm_pair_kernel launch", tmA, tmB, tmC, tmR, p);
  } else {
    st = smem_limit_once(attr_set, ctx.device, block_gemm_kernel<BN, EPI>, C::SMEM,
                         "cudaFuncSetAttribute(block gemm)");
    if (st != HB_OK) return st;
    const int units = m_tiles * n_tiles;
    return launch_pdl(block_gemm_kernel<BN, EPI>, units < ctx.num_sms ? units : ctx.num_sms, kWideThreads, C::SMEM,
                      stream, "block_gemm_kernel launch", tmA, tmB, tmC, tmR, p);
  }
}

template <int NT, int EPI>
hb_status launch_skinny(const DeviceCtx& ctx, const void* A, const void* B, Params p, cudaStream_t stream) {
  using C = CfgSkinny<NT>;
  constexpr bool SWIGLU = EPI == HB_EPI_SWIGLU;
  p.groups = (p.M + NT - 1) / NT;
  int tiles;
  if (SWIGLU) {
    // G gate and G up rows of one 128-row block: as small as the waves that
    // whole blocks take allow
    auto waves = [&](int g) { return (p.N / 128 * (64 / g) * p.groups + ctx.num_sms - 1) / ctx.num_sms; };
    int g = 64;
    while (g > 8 && waves(g / 2) <= waves(g)) g /= 2;
    p.rows = 2 * g;
    tiles = p.N / 128 * (64 / g) * p.groups;
  } else {
    // as few waves as 128-row tiles allow, their rows spread evenly
    const int per_wave = ctx.num_sms / p.groups;  // weight tiles
    const int waves = (p.N + 128 * per_wave - 1) / (128 * per_wave);
    const int even = (p.N + waves * per_wave - 1) / (waves * per_wave);
    p.rows = (even + 7) / 8 * 8;
    tiles = (p.N + p.rows - 1) / p.rows * p.groups;
  }
  const int stage_bytes = 2 * (p.rows + NT) * 128;
  const int avail = 232448 - C::FIXED;
  p.stages = avail / stage_bytes < C::MAX_STAGES ? avail / stage_bytes : C::MAX_STAGES;
  const int smem = C::FIXED + p.stages * stage_bytes;
  CUtensorMap tmA, tmB;
  hb_status st = encode_tmap_2d(&tmA, A, p.K, p.M, p.lda, BK, NT, true, 1);
  if (st != HB_OK) return st;
  st = encode_tmap_2d(&tmB, B, p.K, p.N, p.K, BK, SWIGLU ? p.rows / 2 : p.rows, true, 1);
  if (st != HB_OK) return st;
  static std::atomic<bool> attr_set[kMaxDevices];
  st = smem_limit_once(attr_set, ctx.device, block_gemm_skinny_kernel<NT, EPI>, 232448,
                       "cudaFuncSetAttribute(block gemm skinny)");
  if (st != HB_OK) return st;
  return launch_pdl(block_gemm_skinny_kernel<NT, EPI>, tiles < ctx.num_sms ? tiles : ctx.num_sms, kSkinnyThreads, smem,
                    stream, "block_gemm_skinny_kernel launch", tmA, tmB, p);
}

// Rows of weights of a tile, with groups of nt tokens, if one wave of tiles
// holds the output; 0 if it does not.
template <bool SWIGLU>
int one_wave_rows(const DeviceCtx& ctx, const Params& p, int nt) {
  const int groups = (p.M + nt - 1) / nt;
  if (groups > ctx.num_sms) return 0;
  const int per_wave = ctx.num_sms / groups;  // weight tiles
  if (SWIGLU) {
    int g = 8;
    while (g < 64 && p.N / 128 * (64 / g) > per_wave) g *= 2;
    return p.N / 128 * (64 / g) <= per_wave ? 2 * g : 0;
  }
  const int rows = ((p.N + per_wave - 1) / per_wave + 7) / 8 * 8;
  return rows <= BM ? rows : 0;
}

// Where one wave of tiles of weight rows x 16, 32 or 64 tokens holds the output,
// 256 x 128 tiles would leave most SMs idle: 128 x 4096 x 4096 8.6 us against
// 11.0, 128 x 9728 x 4096 10.9 against 11.9 (SWIGLU with 128 rows 13.1 against
// 12.2: up to 64), 512 x 2400 x 4096 10.1 against 11.2 (measured with the
// weights fetched ahead of the wait).  Of the token counts the
// one whose tile has the fewest rows of weights and tokens to load.  Up to 64
// tokens take such tiles in several waves too.  Else tiles of 128 rows (one
// CTA) or 256 (a pair), by the waves they need and the time of a K block: 286
// ns for 128 x 128, 237 for 256 x 128, 394 for 256 x 256.  All three measured
// (us, in this order; * the rule's): 512 x 4096 x 14336 32.0, 31.5*, 54.8;
// 512 x 4096 x 4096 12.3, 12.7*, 19.7 (both RESIDUAL); 512 x 6144 x 4096 22.8,
// 22.2, 18.7*; 512 x 28672 x 4096 SWIGLU 66.5, 65.7, 52.1*; 1024 x 4096 x 14336
// 62.6, 58.5, 55.5*; 2048 x 4096 x 4096 39.2, 38.3, 36.8*; 4096 x 9216 x 7168
// 232, 225, 190*.
template <int EPI>
hb_status launch_epi(const DeviceCtx& ctx, const void* A, const void* B, const Params& p, cudaStream_t stream) {
  constexpr bool SWIGLU = EPI == HB_EPI_SWIGLU;
  int nt = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 0, best = 0;
  for (int t = 16; t <= 64; t *= 2) {
    const int rows = one_wave_rows<SWIGLU>(ctx, p, t);
    if (rows == 0 || (SWIGLU && rows > 64 && t < p.M) || (best != 0 && rows + t >= best)) continue;
    nt = t;
    best = rows + t;
  }
  if (nt == 16) return launch_skinny<16, EPI>(ctx, A, B, p, stream);
  if (nt == 32) return launch_skinny<32, EPI>(ctx, A, B, p, stream);
  if (nt == 64) return launch_skinny<64, EPI>(ctx, A, B, p, stream);
  // ns of a K block of all waves
  auto time = [&](int ns, int rows, int cols, int slots) {
    const long long tiles = static_cast<long long>((p.M + rows - 1) / rows) * ((p.N + cols - 1) / cols);
    return (tiles + slots - 1) / slots * ns;
  };
  const long long one = time(286, BM, 128, ctx.num_sms), narrow = time(237, 2 * BM, 128, ctx.num_sms / 2);
  const long long broad = time(394, 2 * BM, 256, ctx.num_sms / 2);
  if (p.M <= BM || (one < narrow && one < broad)) return launch_wide<128, EPI, false>(ctx, A, B, p, stream);
  if (narrow < broad) return launch_wide<128, EPI, true>(ctx, A, B, p, stream);
  return launch_wide<256, EPI, true>(ctx, A, B, p, stream);
}

}  // namespace

hb_status gemm_e4m3_block_launch(const DeviceCtx& ctx, const void* A, int lda, const float* sa, const void* B,
                                 const float* sb, void* C, int ldc, const void* R, int M, int N, int K, int epi,
                                 cudaStream_t stream, bool weights_ready) {
  Params p = {};
  p.preload = weights_ready;
  p.M = M;
  p.N = N;
  p.K = K;
  p.lda = lda;
  p.C = C;
  p.R = R;
  p.ldc = ldc;
  p.out_cols = epi == HB_EPI_SWIGLU ? N / 2 : N;
  p.sa = sa;
  p.sb = sb;
  p.f_blocks = (N / 2 + 127) / 128;
  p.kblocks = (K + BK - 1) / BK;
  p.status = ctx.status;
  switch (epi) {
    case HB_EPI_STORE: return launch_epi<HB_EPI_STORE>(ctx, A, B, p, stream);
    case HB_EPI_RESIDUAL: return launch_epi<HB_EPI_RESIDUAL>(ctx, A, B, p, stream);
    case HB_EPI_SWIGLU: return launch_epi<HB_EPI_SWIGLU>(ctx, A, B, p, stream);
    default: return launch_epi<HB_EPI_F32>(ctx, A, B, p, stream);
  }
}

}  // namespace hb

extern "C" hb_status hb_gemm_e4m3_block(const void* A, const float* s_a, const void* B, const float* s_b, void* C,
                                        const void* R, int32_t M, int32_t N, int32_t K, int32_t epilogue,
                                        void* stream) {
  hb::clear_error();
  HB_REQUIRE(A && s_a && B && s_b && C, "hb_gemm_e4m3_block: null operand");
  HB_REQUIRE(M >= 1 && N >= 8 && K >= 16, "hb_gemm_e4m3_block: bad shape M=%d N=%d K=%d", M, N, K);
  HB_REQUIRE(M <= 1 << 30 && N <= 1 << 30 && K <= 1 << 30, "hb_gemm_e4m3_block: sizes up to 2^30");
  HB_REQUIRE(K % 16 == 0 && N % 8 == 0, "hb_gemm_e4m3_block: K %% 16 and N %% 8 required (K=%d N=%d)", K, N);
  HB_REQUIRE(epilogue >= HB_EPI_STORE && epilogue <= HB_EPI_F32, "hb_gemm_e4m3_block: unknown epilogue %d", epilogue);
  HB_REQUIRE(epilogue != HB_EPI_SWIGLU || N % 128 == 0, "hb_gemm_e4m3_block: SWIGLU needs N %% 128 == 0");
  HB_REQUIRE(epilogue != HB_EPI_RESIDUAL || R != nullptr, "hb_gemm_e4m3_block: RESIDUAL needs R");
  HB_REQUIRE(hb::aligned16(A) && hb::aligned16(B) && hb::aligned16(C) && (R == nullptr || hb::aligned16(R)),
             "hb_gemm_e4m3_block: operands must be 16-byte aligned");
  HB_REQUIRE(hb::aligned4(s_a) && hb::aligned4(s_b), "hb_gemm_e4m3_block: scales must be 4-byte aligned");
  hb::DeviceCtx ctx;
  hb_status st = hb::device_context(&ctx);
  if (st != HB_OK) return st;
  const int ldc = epilogue == HB_EPI_SWIGLU ? N / 2 : N;
  // whatever is ahead on the stream may have written B
  return hb::gemm_e4m3_block_launch(ctx, A, K, s_a, B, s_b, C, ldc, R, M, N, K, epilogue,
                                    static_cast<cudaStream_t>(stream), false);
}
