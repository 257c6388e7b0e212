// Attention of prompt chunks over a cache of E4M3 codes, on the
// 5th-generation tensor cores.
//
// A chunk's query at position p attends to keys 0..p of its request
// (Sarathi-Serve reading notes, sections 3.1 and 7.5b):
//   S = Q K^T, P = 2^(S scale - m), O += P V, out = O / sum P,
// K = 2^ek codes and V = 2^ev codes widened to bf16, which is exact (powers of
// two), so the products are those of hb_attention with such a cache in bf16.
//
// Every 128 rows and q head go over the same K and V again, so the codes are
// widened once, by a kernel ahead (widen_kernel), into scratch of the workspace
// laid out for whole-block copies.  That scratch is bounded (kScratchKeys);
// sequences behind its end are widened block by block beside the MMAs instead
// (WIDEN: the same kernel with five more warps, whose 16 at 128 registers spill 544
// bytes), which takes 3.7 times as long.
//
// The tensor pipe bounds it, 4 d_head FLOP a pair and q head: 2048 rows behind
// 14336 keys, 56 q heads on 8 of 128, 578 us back to back with the widening, under
// the power limit (floor 466 at cuBLAS's burst rate, 520 at its sustained one);
// alone the kernel takes 550, the pipe 73% active.  With two tiles a CTA and one
// set of S columns each, so that a tile's next S waits for its PV, 701.
//
// Unit: a 128-row tile of one q head, and keys 0 .. last in blocks of 128.
// Tensor memory holds O and three sets of S columns: block G of the CTA has set
// G % 3, P is written over its S.  So the S of two blocks ahead is computed while
// one block is in its softmax and another in its PV.
//
// The keys of a short chunk behind a long prefix are split (part_count), a unit a
// part: 6 rows behind 10610 keys, 12 q heads on 4 of 64, 61 us
// whole and 28 in 8 parts, with the widening and the join.
//
// Warp roles (one CTA per SM):
//   warp 0      finds the unit (its lanes scan the sequences), publishes it in
//               shared memory, loads its Q tile and the K and V blocks;
//   warp 1      S = Q K_j^T (M = N = 128) into the set's columns;
//   warp 10     O += P V_j with P read from the same columns (bf16, written over
//               S).  Two issuing warps, because a wait costs an issuer some 100
//               clocks even where it ends at once;
//   warps 2-5, 6-9  softmax of every other block: a thread has one row and takes
//               its 128 scores into registers.  A row's maximum goes from group to
//               group through shared memory, block by block, ahead of the
//               exponentials, which are most of the work; each group keeps the sum
//               of its own blocks.  O is rescaled only where a row's maximum grew
//               by more than 2^8.  The group of a unit's last block stores O / l.
// WIDEN: warp 0 loads K codes, 64 keys a slot, into a ring, warp 15 does so with
// V's; scale bytes, 16 a page, go through their registers a block ahead (a copy
// costs the issuing warp some 150 clocks).  Warps 11-14 widen: a warp takes one
// 16-key page of a slot, 16 codes a lane at a time, into the 128-byte swizzled K
// or V block.
//
// Keys behind a sequence's last become zeros.  A value whose scale is NaN must
// reach the rows that see its key and no other: 0 * NaN would spread it, so the
// widening puts the NaN into the key's K row (S is masked by selection) and
// zeros into V.
// Every wait is bounded; an expired wait sets the status word and unwinds.
#include "attention_e4m3.cuh"
#include "attention_tc.cuh"

namespace hb {
namespace {

using namespace dev;
using kv8::first_tile_blocks;
using kv8::mul_bf16x2;
using kv8::Params;
using kv8::part_count;
using kv8::part_floats;
using kv8::part_row;
using tc::mma_bf16_ts;
using tc::smem_desc_sw128_mn;
using tc::tmem_st_wait;

constexpr int TQ = 128, TK = 128;
constexpr int HK = 64;  // keys of a ring slot
constexpr int kSoft0 = 2, kPv = 10, kConv0 = 11, kConvWarps = 4, kVWarp = 15;
template <bool WIDEN>
constexpr int kThreads = 32 * (WIDEN ? kVWarp + 1 : kConv0);
constexpr float kRescale = 8.0f;

struct Unit {
  int valid, seq, g, nblk;
  int row;  // of the scratch: key 0 of this sequence and kv head
  int row0, nrows, pos0, head;
  int part_row;
  int page0, part;  // a part of the keys: row and pos0 count from its first key, in page page0 of the
                    // sequence; part -1: all keys
};
constexpr int SETS = 3;  // of S and P columns: block G of the CTA has set G % 3

template <int D, bool WIDEN>
struct TC {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_TILE = 128 * 128;        // 128 rows x 128 bytes (64 dims)
  static constexpr int TILE = HALVES * HALF_TILE;    // a Q tile, a K or V block
  static constexpr int KST = WIDEN ? 2 : 3, VST = KST;    // blocks in flight
  static constexpr int SLOTS = WIDEN ? (D == 128 ? 2 : 4) : 0;  // of the K and of the V code ring
  static constexpr int SLOT = HK * D;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = TILE;
  static constexpr int OFF_V = OFF_K + KST * TILE;
  static constexpr int OFF_C = OFF_V + VST * TILE;
  static constexpr int OFF_S = OFF_C + 2 * SLOTS * SLOT;  // scales: K's (or V's) 64 bytes, V's 64 bytes beside K
  static constexpr int OFF_U = OFF_S + 2 * SLOTS * 2 * HK;
  static constexpr int OFF_M = OFF_U + 96;           // a row's maximum, from block to block
  static constexpr int OFF_L = OFF_M + TQ * 4;       // [2] a row's sum over the other group's blocks
  static constexpr int OFF_BAR = OFF_L + 2 * TQ * 4;
  static constexpr int SMEM = OFF_BAR + (44 + 4 * SLOTS) * 8 + 8 + 1024;
  static_assert(2 * sizeof(Unit) <= 96 && OFF_BAR % 8 == 0 && SMEM <= 232448, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;  // S0 S1 S2 (P over them) O
};

// bf16 factors of a scale byte b: code * 2^-120 times `first` times `second` is
// code * 2^(b - 127).  2^(120 + e) is no bf16 number from e = 8 on.
struct Factor {
  uint32_t first, second;
};
__device__ __forceinline__ Factor factor_of(uint32_t b) {
  const uint32_t f = b == 255 ? 0x7fc0u : b <= 134 ? (b + 120) << 7 : 0x7f00u;
  const uint32_t s = b == 255 || b <= 134 ? 0x3f80u : (b - 7) << 7;
  return {f * 0x10001u, s * 0x10001u};
}

__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_u8(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void sts_u4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 16 codes as bf16 in their order, times 2^120 * factor.  The fields are moved
// by two multiply-adds where shifts and masks would do it in three (codes_moved):
// with x = two codes in the lower byte of each half, x * 16 has exponent and
// mantissa in place and the sign at bit 11, and sign * (256 - 16) takes that to
// bit 15.  The widening shares its SM with the softmax, and the multiplier is
// the less busy pipe.
__device__ __forceinline__ uint32_t codes_moved_low(uint32_t x) { return (x & 0x00800080u) * 240u + x * 16u; }
__device__ __forceinline__ void widen16(const uint4& raw, uint32_t factor, uint32_t (&o)[8]) {
  const uint32_t word[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[2 * e] = mul_bf16x2(codes_moved_low(__byte_perm(word[e], 0, 0x4140)), factor);
    o[2 * e + 1] = mul_bf16x2(codes_moved_low(__byte_perm(word[e], 0, 0x4342)), factor);
  }
}

// tcgen05.wait::ld that the loaded registers depend on
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The tile that is the i-th of its kv head, heaviest rows first.
__device__ __forceinline__ void tile_of(const Params& p, int i, int ntiles, int q0, int qlen, int kvl, Unit& w) {
  const int rt = ntiles - 1 - i / p.grp;
  w.head = w.g * p.grp + i % p.grp;
  w.row0 = q0 + rt * TQ;
  w.nrows = min(TQ, qlen - rt * TQ);
  w.pos0 = kvl - qlen + rt * TQ;
  w.nblk = (w.pos0 + w.nrows + TK - 1) / TK;
}

// keys of a sequence in the scratch: whole blocks
__device__ __forceinline__ int padded(int kvl) { return (kvl + TK - 1) / TK * TK; }

// Which of this kernel's sequences (those of several rows) an item falls into,
// sequence by sequence in order, by a whole warp; items ascend from call to call.
// count(qlen, kvl, base): items of a sequence whose scratch starts at key `base`.
// Sequences out of range are reported and have no items (and no scratch).
struct SeqScan {
  int s0 = 0, items = 0, keys = 0;  // of the sequences ahead of s0
  int seq, q0, qlen, kvl;           // the one found
  template <typename Count>
  __device__ __forceinline__ bool find(const Params& p, int v, int lane, Count count, int* local, int* base) {
    while (s0 < p.S) {
      const int s = s0 + lane;
      int c = 0, k = 0, a = 0, ql = 0, kl = 0;
      if (s < p.S) {
        a = ld_s32(p.q_start + s);
        const int q1 = ld_s32(p.q_start + s + 1);
        ql = q1 - a;
        kl = ld_s32(p.kv_len + s);
        if (a < 0 || q1 > p.T || ql < 1 || kl < ql || kl > p.max_kv_len || (kl + 15) / 16 > p.max_pages)
          flag_error(p.status, kStatusIndex);
        else if (ql > 1 || p.no_decodes)
          k = padded(kl);
      }
      int kend = k;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, kend, o);
        if (lane >= o) kend = min(kend + u, 1 << 29);  // (far behind any scratch: no overflow)
      }
      kend = min(kend + keys, 1 << 29);
      if (k > 0) c = count(ql, kl, kend - k);
      int end = c;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += u;
      }
      end += items;
      const unsigned at = __ballot_sync(0xffffffffu, v < end);
      if (at != 0) {
        const int l = __ffs(static_cast<int>(at)) - 1;
        seq = s0 + l;
        *local = v - __shfl_sync(0xffffffffu, end - c, l);
        *base = __shfl_sync(0xffffffffu, kend - k, l);
        q0 = __shfl_sync(0xffffffffu, a, l);
        qlen = __shfl_sync(0xffffffffu, ql, l);
        kvl = __shfl_sync(0xffffffffu, kl, l);
        return true;
      }
      items = __shfl_sync(0xffffffffu, end, 31);
      keys = __shfl_sync(0xffffffffu, kend, 31);
      s0 += 32;
    }
    return false;
  }
};

// The codes of several-row sequences as bf16, key after key of each kv head, to
// whole 128-key blocks; a warp takes one page of one kv head.
template <int D>
__global__ void __launch_bounds__(256) widen_kernel(Params p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int PIECES = D / 16, KEYS = 32 / PIECES, STEPS = 16 / KEYS;
  const int lane = threadIdx.x & 31, c = lane % PIECES;
  SeqScan scan;
  // neighbouring items on different SMs
  for (int v = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;; v += 8 * gridDim.x) {
    int local, base;
    if (!scan.find(p, v, lane, [&](int, int kvl, int at) {
          return at + padded(kvl) <= p.scratch_keys ? padded(kvl) / 16 * p.n_kv : 0;
        }, &local, &base))
      return;
    const int g = local % p.n_kv, pg = local / p.n_kv, live = scan.kvl - pg * 16;
    uint4 k[STEPS], w[STEPS];
    uint32_t kb[STEPS], vb[STEPS];
    size_t at = 0;
    if (live > 0) {
      int id = ld_s32(p.block_table + static_cast<size_t>(scan.seq) * p.max_pages + pg);
      if (id < 0 || id >= p.num_pages) {
        flag_error(p.status, kStatusIndex);
        id = 0;
      }
      at = (static_cast<size_t>(id) * p.n_kv + g) * 16;
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = i * KEYS + lane / PIECES;
      k[i] = w[i] = make_uint4(0, 0, 0, 0);
      kb[i] = vb[i] = 127;
      if (r < live) {
        k[i] = ld_u4(p.k + (at + r) * D + c * 16);
        w[i] = ld_u4(p.v + (at + r) * D + c * 16);
        kb[i] = ld_u8(p.ks + at + r);
        vb[i] = ld_u8(p.vs + at + r);
      }
    }
    const size_t row = static_cast<size_t>(base) * p.n_kv + static_cast<size_t>(g) * padded(scan.kvl) + pg * 16;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const size_t to = (row + i * KEYS + lane / PIECES) * D + c * 16;
      const Factor fk = factor_of(vb[i] == 255 ? 255 : kb[i]);
      Factor fv = factor_of(vb[i]);
      if (vb[i] == 255) fv = {0u, 0x3f803f80u};
      uint32_t o[8];
      widen16(k[i], fk.first, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(o[e], fk.second);
      uint4* dst = reinterpret_cast<uint4*>(p.scratch_k + to);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      widen16(w[i], fv.first, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(o[e], fv.second);
      dst = reinterpret_cast<uint4*>(p.scratch_v + to);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <int D, bool WIDEN>
__global__ void __launch_bounds__(kThreads<WIDEN>, 1)
    chunk_e4m3_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, Params p) {
  using C = TC<D, WIDEN>;
  // The decode kernel behind this one runs beside it.  Its inputs are there: the
  // widening's CTAs had waited for all that is ahead before this kernel could start.
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sC = smem + C::OFF_C;
  uint8_t* sS = smem + C::OFF_S;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* u_full = bar;            // [2] unit published
  uint64_t* u_empty = bar + 2;       // [2] V's producer, the MMA, softmax and widening warps have read it
  uint64_t* q_full = bar + 4;
  uint64_t* q_empty = bar + 5;
  uint64_t* k_full = bar + 8;        // [KST] block landed, or widening warps
  uint64_t* k_empty = bar + 11;      // [KST]
  uint64_t* v_full = bar + 14;       // [VST]
  uint64_t* v_empty = bar + 17;
  uint64_t* s_full = bar + 20;       // [SETS]
  uint64_t* p_full = bar + 23;       // [SETS] four softmax warps
  uint64_t* pv_done = bar + 26;      // [SETS]
  uint64_t* o_empty = bar + 29;      // four softmax warps
  uint64_t* drain = bar + 30;        // [issuer]
  uint64_t* m_full = bar + 32;       // [quarter] a block's maximum is known
  uint64_t* l_full = bar + 36;       // [2][quarter] the other group's sums are there
  uint64_t* c_full = bar + 44;       // [2 SLOTS] codes landed, scales stored: K's ring, then V's
  uint64_t* c_empty = c_full + 2 * C::SLOTS;  // [2 SLOTS] widening warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 44 + 4 * C::SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Unit* units = reinterpret_cast<Unit*>(smem + C::OFF_U);  // [2]

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], 2 + 8 + (WIDEN ? kConvWarps + 1 : 0));
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < C::KST; ++i) {
      mbar_init(&k_full[i], WIDEN ? kConvWarps : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::VST; ++i) {
      mbar_init(&v_full[i], WIDEN ? kConvWarps : 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < SETS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&m_full[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&l_full[i], 1);
    for (int i = 0; i < 2 * C::SLOTS; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], kConvWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_empty, 4);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // unit n of this CTA, read from slot n % 2 by a whole warp
  auto next_unit = [&](int n, Unit& w) {
    const bool got = mbar_wait(&u_full[n & 1], (n >> 1) & 1, abort_flag, p.status);
    if (!__all_sync(0xffffffffu, got)) return false;
    w = units[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[n & 1]);
    return w.valid != 0;
  };

  // the K or V codes of a unit's blocks into their ring, by a whole warp
  constexpr int kSlots = WIDEN ? C::SLOTS : 1;
  int half = 0;  // 64-key halves loaded so far
  auto load_codes = [&](const Unit& w, bool is_v) {
    const int* bt = p.block_table + static_cast<size_t>(w.seq) * p.max_pages + w.page0;
    const int npages = (w.pos0 + w.nrows + 15) / 16;
    uint64_t* full = c_full + (is_v ? C::SLOTS : 0);
    uint64_t* empty = c_empty + (is_v ? C::SLOTS : 0);
    uint8_t* codes = sC + (is_v ? C::SLOTS * C::SLOT : 0);
    uint8_t* scales = sS + (is_v ? C::SLOTS * 2 * HK : 0);
    // lane l < 8 has row, of 16 in the pool, of page l of a block: the id loaded
    // three blocks ahead, the scales one ahead
    auto load_id = [&](int j) { return lane < 8 && j * 8 + lane < npages ? ld_s32(bt + j * 8 + lane) : 0; };
    auto row_of = [&](int id) {
      if (id < 0 || id >= p.num_pages) {
        flag_error(p.status, kStatusIndex);
        id = 0;
      }
      return (id * p.n_kv + w.g) * 16;
    };
    auto load_scale = [&](const uint8_t* base, int j, int row) {
      return lane < 8 && j * 8 + lane < npages ? ld_u4(base + row) : make_uint4(0, 0, 0, 0);
    };
    int row = row_of(load_id(0)), id1 = load_id(1), id2 = load_id(2);
    uint4 s0 = load_scale(is_v ? p.vs : p.ks, 0, row), s1 = make_uint4(0, 0, 0, 0);
    if (!is_v) s1 = load_scale(p.vs, 0, row);
    for (int j = 0; j < w.nblk; ++j) {
      const int row1 = row_of(id1), id3 = load_id(j + 3);
      const uint4 n0 = load_scale(is_v ? p.vs : p.ks, j + 1, row1);
      const uint4 n1 = is_v ? n0 : load_scale(p.vs, j + 1, row1);
#pragma unroll 1
      for (int i = 0; i < 2; ++i, ++half) {
        const int slot = half % kSlots;
        const bool free = mbar_wait(&empty[slot], ((half / kSlots) & 1) ^ 1u, abort_flag, p.status);
        if (!__all_sync(0xffffffffu, free)) return false;
        const int here = max(0, min(4, npages - j * 8 - i * 4)), l4 = lane & 3;
        const bool mine = lane < 8 && (lane >> 2) == i && l4 < here;
        if (mine) {
          *reinterpret_cast<uint4*>(scales + slot * 2 * HK + l4 * 16) = s0;
          if (!is_v) *reinterpret_cast<uint4*>(scales + slot * 2 * HK + HK + l4 * 16) = s1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], here * 16 * D);
        __syncwarp();
        if (mine) tma_load_2d(codes + slot * C::SLOT + l4 * 16 * D, is_v ? &tmV : &tmK, &full[slot], 0, row);
      }
      row = row1;
      id1 = id2;
      id2 = id3;
      s0 = n0;
      s1 = n1;
    }
    return true;
  };
  // the widened K and V blocks of a unit, by one thread: K's two ahead, as S is
  int k_blocks = 0, v_blocks = 0;  // loaded so far
  auto load_blocks = [&](const Unit& w) {
    for (int j = -2; j < w.nblk; ++j) {
      if (j + 2 < w.nblk) {
        const int st = k_blocks % C::KST, row = w.row + (j + 2) * TK;
        if (!mbar_wait(&k_empty[st], ((k_blocks / C::KST) & 1) ^ 1u, abort_flag, p.status)) return false;
        mbar_arrive_expect_tx(&k_full[st], C::TILE);
#pragma unroll
        for (int hf = 0; hf < C::HALVES; ++hf)
          tma_load_2d(sK + st * C::TILE + hf * C::HALF_TILE, &tmK, &k_full[st], hf * 64, row);
        ++k_blocks;
      }
      if (j >= 0) {
        const int st = v_blocks % C::VST, row = w.row + j * TK;
        if (!mbar_wait(&v_empty[st], ((v_blocks / C::VST) & 1) ^ 1u, abort_flag, p.status)) return false;
        mbar_arrive_expect_tx(&v_full[st], C::TILE);
#pragma unroll
        for (int hf = 0; hf < C::HALVES; ++hf)
          tma_load_2d(sV + st * C::TILE + hf * C::HALF_TILE, &tmV, &v_full[st], hf * 64, row);
        ++v_blocks;
      }
    }
    return true;
  };
  // A copying warp leaves once its copies have landed, whichever warp's wait expires
  // meanwhile: it waits for the last ones as their readers do, and after an expired
  // wait for a while more (bounded).
  int q_tiles = 0;  // loaded so far
  auto land_copies = [&](bool ok) {
    if (lane != 0) return;
    auto land = [&](uint64_t* full, int use) {
      ok = ok && mbar_wait(full, use & 1, abort_flag, p.status);
      if (!ok) mbar_drain(full, use & 1);
    };
    if (q_tiles > 0) land(q_full, q_tiles - 1);
    if (!WIDEN) {
      for (int b = max(0, k_blocks - C::KST); b < k_blocks; ++b) land(&k_full[b % C::KST], b / C::KST);
      for (int b = max(0, v_blocks - C::VST); b < v_blocks; ++b) land(&v_full[b % C::VST], b / C::VST);
      return;
    }
    uint64_t* full = c_full + (warp == kVWarp ? kSlots : 0);
    for (int h = max(0, half - kSlots); h < half; ++h) land(&full[h % kSlots], h / kSlots);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producers
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    SeqScan scan;
    bool ok = true;
    for (int n = 0, v = blockIdx.x; ok; ++n, v += gridDim.x) {
      // the sequence that unit v falls into
      Unit w;
      int local, base;
      w.valid = scan.find(p, v, lane, [&](int qlen, int kvl, int at) {
        const bool fits = at + padded(kvl) <= p.scratch_keys;
        const int units = p.n_q * ((qlen + TQ - 1) / TQ);
        return fits != WIDEN ? units * part_count(units, first_tile_blocks(qlen, kvl)) : 0;
      }, &local, &base);
      if (w.valid) {
        const int ntiles = (scan.qlen + TQ - 1) / TQ;
        w.seq = scan.seq;
        w.g = local % p.n_kv;
        w.row = base * p.n_kv + w.g * padded(scan.kvl);
        const int blocks = first_tile_blocks(scan.qlen, scan.kvl), parts = part_count(p.n_q * ntiles, blocks);
        const int i = local / p.n_kv;
        tile_of(p, i / parts, ntiles, scan.q0, scan.qlen, scan.kvl, w);
        w.part = -1;
        w.page0 = 0;
        if (parts > 1) {
          w.part = i % parts;
          w.part_row = part_row(p, w.row0, scan.seq, scan.q0);
          const int per = blocks / parts, first = w.part * per;
          w.nblk = w.part == parts - 1 ? w.nblk - first : per;
          w.row += first * TK;
          w.pos0 -= first * TK;
          w.page0 = first * (TK / 16);
        }
      }
      if (lane == 0) {
        ok = mbar_wait(&u_empty[n & 1], ((n >> 1) & 1) ^ 1u, abort_flag, p.status);
        if (ok) {
          units[n & 1] = w;
          mbar_arrive(&u_full[n & 1]);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) ok = false;
      if (!ok || !w.valid) break;
      if (lane == 0) {
        ok = mbar_wait(q_empty, (n & 1) ^ 1u, abort_flag, p.status);
        if (ok) {
          mbar_arrive_expect_tx(q_full, C::TILE);
#pragma unroll
          for (int hf = 0; hf < C::HALVES; ++hf)
            tma_load_3d(sQ + hf * C::HALF_TILE, &tmQ, q_full, hf * 64, w.head, w.row0);
          ++q_tiles;
        }
      }
      if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) {
        ok = false;
        break;
      }
      if (WIDEN) {
        ok = load_codes(w, false);
      } else {
        if (lane == 0) ok = load_blocks(w);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
    }
    land_copies(ok);
  } else if (WIDEN && warp == kVWarp) {
    bool ok = true;
    Unit w;
    for (int n = 0; ok && next_unit(n, w); ++n) ok = load_codes(w, true);
    land_copies(ok);
  } else if (warp == 1 || warp == kPv) {
    // ------------------------------------------------------------ MMA issuers
    // The whole warp walks the loop and one elected lane issues: in a single-lane
    // branch every descriptor would be moved to a uniform register anew.
    int G = 0;  // blocks so far
    bool ok = true;
    Unit w;
    auto wait = [&](uint64_t* bar, int parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_at(smem_u32(bar), parity, abort_flag, p.status));
    };
    if (warp == 1) {
      constexpr uint32_t idS = idesc_bf16_f32(TQ, TK);
      const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ)), k_desc = smem_desc_sw128(smem_u32(sK));
      for (int n = 0; ok && next_unit(n, w); ++n) {
        wait(q_full, n & 1);
#pragma unroll 1
        for (int j = 0; j < w.nblk && ok; ++j, ++G) {
          const int st = G % C::KST, set = G % SETS;
          wait(&k_full[st], (G / C::KST) & 1);
          wait(&pv_done[set], ((G / SETS) & 1) ^ 1);  // S is written over the set's last P
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = k_desc + ((st * C::TILE) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * C::HALF_TILE + (kk & 3) * 32) >> 4;
              mma_bf16(tmem + set * 128, q_desc + off, kd + off, idS, kk > 0 ? 1u : 0u);
            }
            mma_commit(&s_full[set]);
            mma_commit(&k_empty[st]);
            if (j == w.nblk - 1) mma_commit(q_empty);
          }
          __syncwarp();
        }
      }
    } else {
      constexpr uint32_t idPV = idesc_bf16_f32(TQ, D) | (1u << 16);  // B (V) is MN-major
      const uint64_t v_desc = smem_desc_sw128_mn(smem_u32(sV), C::HALF_TILE, 1024);
      const uint32_t tO = tmem + SETS * 128;
      for (int n = 0; ok && next_unit(n, w); ++n) {
        wait(o_empty, (n & 1) ^ 1);
#pragma unroll 1
        for (int j = 0; j < w.nblk && ok; ++j, ++G) {
          const int st = G % C::VST, set = G % SETS;
          wait(&v_full[st], (G / C::VST) & 1);
          wait(&p_full[set], (G / SETS) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc + ((st * C::TILE) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < TK / 16; ++kk)
              mma_bf16_ts(tO, tmem + set * 128 + kk * 8, vd + ((kk * 2048) >> 4), idPV, (j > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&pv_done[set]);
            mma_commit(&v_empty[st]);
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) {
      // nothing may still read shared memory or write tensor memory at the end, where
      // another warp's wait has expired too
      uint64_t* done = &drain[warp == 1 ? 0 : 1];
      mma_commit(done);
      mbar_drain(done, 0);
    }
  } else if (WIDEN && warp >= kConv0) {
    // ------------------------------------------------------------ widening
    const int pg = warp - kConv0;  // page of a slot
    constexpr int PIECES = D / 16;             // 16-code pieces of a key
    constexpr int STEPS = 16 * PIECES / 32;    // pieces of a lane
    constexpr int KEYS = 32 / PIECES;          // keys of a warp's step
    const int c = lane % PIECES, key0 = pg * 16 + lane / PIECES;  // this lane's first key of the half
    // 16 dims are two 16-byte chunks of the key's row in their 64-dim half.
    // Lanes of the upper half store theirs in the other order: the eight lanes
    // that a store takes at a time then meet eight different bank groups.
    const int flip = c >> 2;
    const uint32_t col = (c >> 2) * C::HALF_TILE;
    const int j0 = 2 * (c & 3) + flip, j1 = 2 * (c & 3) + (flip ^ 1);
    int J = 0;
    bool ok = true;
    Unit w;
    for (int n = 0; ok && next_unit(n, w); ++n) {
      const int key_end = w.pos0 + w.nrows;
      for (int j = 0; j < w.nblk && ok; ++j, ++J) {
        const int st = J % 2, use = J / 2;
#pragma unroll 1
        for (int i4 = 0; i4 < 4; ++i4) {  // K keys 0..63, 64..127, V the same
          const int kv = i4 >> 1, hf = i4 & 1;
          const int at = J * 2 + hf, slot = at % kSlots + kv * kSlots;
          bool landed = mbar_wait(&c_full[slot], (at / kSlots) & 1, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, landed)) {
            ok = false;
            break;
          }
          const uint32_t codes = smem_u32(sC + slot * C::SLOT) + key0 * D + c * 16;
          const uint32_t scales = smem_u32(sS + slot * 2 * HK) + key0;
          uint4 raw[STEPS];
          uint32_t sb[STEPS];
          bool plain = j * TK + (hf + 1) * HK <= key_end;
#pragma unroll
          for (int i = 0; i < STEPS; ++i) {
            raw[i] = lds_u4(codes + i * KEYS * D);
            sb[i] = lds_u8(scales + i * KEYS);
            // a value's NaN goes into its key
            if (kv == 0 && lds_u8(scales + HK + i * KEYS) == 255) sb[i] = 255;
            plain &= sb[i] <= 134;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&c_empty[slot]);
          bool free = mbar_wait(kv ? &v_empty[st] : &k_empty[st], (use & 1) ^ 1u, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, free)) {
            ok = false;
            break;
          }
          const uint32_t dst = smem_u32((kv ? sV : sK) + st * C::TILE) + col;
          auto put = [&](int i, const uint32_t (&o)[8]) {
            const int r = hf * HK + key0 + i * KEYS;  // key of the block
            const uint32_t row = dst + r * 128;
            const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
            sts_u4(row + ((j0 ^ (r & 7)) << 4), flip ? hi : lo);
            sts_u4(row + ((j1 ^ (r & 7)) << 4), flip ? lo : hi);
          };
          if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
              uint32_t o[8];
              widen16(raw[i], ((sb[i] + 120) << 7) * 0x10001u, o);
              put(i, o);
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < STEPS; ++i) {
              Factor f = factor_of(sb[i]);
              if (j * TK + hf * HK + key0 + i * KEYS >= key_end || (kv == 1 && sb[i] == 255)) f = {0u, 0x3f803f80u};
              uint32_t o[8];
              widen16(raw[i], f.first, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(o[e], f.second);
              put(i, o);
            }
          }
          if (hf == 0) continue;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv ? &v_full[st] : &k_full[st]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int group = (warp - kSoft0) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t tT = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t tO = tT + SETS * 128;
    volatile float* m_row = reinterpret_cast<float*>(smem + C::OFF_M) + r;
    volatile float* l_row = reinterpret_cast<float*>(smem + C::OFF_L) + r;
    int J = 0;     // blocks of the units before
    int both = 0;  // units before of both groups
    Unit w;
    for (int n = 0; next_unit(n, w); ++n) {
      const int lim = r < w.nrows ? w.pos0 + r : w.pos0 + w.nrows - 1;  // last key this row sees
      float m_used = -INFINITY, m_in = -INFINITY, l = 0.f;
      bool ok = true;
#pragma unroll 1
      for (int j = (group ^ J) & 1; j < w.nblk; j += 2) {
        const int G = J + j, set = G % SETS;
        const uint32_t tS = tT + set * 128;
        bool sok = mbar_wait(&s_full[set], (G / SETS) & 1, abort_flag, p.status);
        if (!__all_sync(0xffffffffu, sok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int seen = lim - j * TK;  // columns 0 .. seen of the block
        const bool cut = __any_sync(0xffffffffu, seen < TK - 1);
        uint32_t v[4][32];
        float mp[4];
        tmem_ld_32x32b_x32(tS, v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait32(v[c]);
          if (c < 3) tmem_ld_32x32b_x32(tS + (c + 1) * 32, v[(c + 1) & 3]);
          if (cut) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[c][e] = c * 32 + e <= seen ? v[c][e] : 0xff800000u;
          }
          mp[c] = __uint_as_float(v[c][0]);
#pragma unroll
          for (int e = 1; e < 31; e += 2)
            mp[c] = fmaxf(mp[c], fmaxf(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])));
          mp[c] = fmaxf(mp[c], __uint_as_float(v[c][31]));
        }
        const float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * p.scale_log2;
        // the last block's maximum, from the other group; of the last unit it only
        // keeps the groups in step
        if (G > 0) {
          bool mok = mbar_wait(&m_full[quarter], (G - 1) & 1, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, mok)) {
            ok = false;
            break;
          }
          if (j > 0) m_in = *m_row;
        }
        const bool raise = mx > m_in + kRescale;
        const float m_new = raise ? mx : m_in;
        *m_row = m_new;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m_full[quarter]);
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
          const float alpha = raise ? ex2_approx(m_in - m_new) : 1.f;
          bool lok = mbar_wait(&pv_done[(G - 1) % SETS], ((G - 1) / SETS) & 1, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, lok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t ov[16];
            tmem_ld_32x32b_x16(tO + c, ov);
            tmem_ld_wait16(ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st_32x32b_x16(tO + c, ov);
          }
        }
        if (m_new != m_used) {
          l *= ex2_approx(m_used - m_new);
          m_used = m_new;
        }
        const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
        const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2), neg2 = pack_f32x2(neg_m, neg_m);
        uint64_t rs[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = unpack_f32x2(
                fma_f32x2(pack_f32x2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])), scale2, neg2));
            const float a0 = ex2_approx(y.x), a1 = ex2_approx(y.y);
            rs[e & 1] = add_f32x2(rs[e & 1], pack_f32x2(a0, a1));
            pk[e] = pack_bf16x2(a0, a1);
          }
          tmem_st_32x32b_x16(tS + c * 16, pk);  // over S, which is in registers
        }
        const float2 r2 = unpack_f32x2(add_f32x2(rs[0], rs[1]));
        l += r2.x + r2.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[set]);
      }
      if (!ok) break;
      // the group of the last block stores the rows, with the other's sums
      const int last = J + w.nblk - 1, slot = both & 1;
      J += w.nblk;
      if (w.nblk > 1) {
        if ((last & 1) != group) {
          l_row[slot * TQ] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_full[slot * 4 + quarter]);
        } else {
          bool lok = mbar_wait(&l_full[slot * 4 + quarter], (both >> 1) & 1, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, lok)) break;
          const float other = l_row[slot * TQ];
          l += m_in == m_used ? other : other * ex2_approx(m_in - m_used);
        }
        ++both;
      }
      if ((last & 1) != group) continue;
      bool pok = mbar_wait(&pv_done[last % SETS], (last / SETS) & 1, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, pok)) break;
      tc_fence_after();
      if (w.part >= 0) {
        float* rec = p.chunk_partials +
                     ((static_cast<size_t>(w.part_row + r) * p.n_q + w.head) * p.max_parts + w.part) * part_floats(D);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t ov[32];
          tmem_ld_32x32b_x32(tO + c, ov);
          tmem_ld_wait32(ov);
          if (r < w.nrows)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(rec + c + 4 * i) = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
        }
        if (r < w.nrows) *reinterpret_cast<float2*>(rec + D) = make_float2(m_used, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty);  // O was read into registers
        continue;
      }
      const float inv = 1.f / l;
      __nv_bfloat16* orow = p.out + (static_cast<size_t>(w.row0 + r) * p.n_q + w.head) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t ov[32];
        tmem_ld_32x32b_x32(tO + c, ov);
        tmem_ld_wait32(ov);
        if (r < w.nrows) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t q4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              q4[e] = pack_bf16x2(__uint_as_float(ov[8 * i + 2 * e]) * inv, __uint_as_float(ov[8 * i + 2 * e + 1]) * inv);
            dst[i] = make_uint4(q4[0], q4[1], q4[2], q4[3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);  // O was read into registers
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool WIDEN>
hb_status launch_chunk(const DeviceCtx& ctx, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                       const Params& p, int grid, cudaStream_t stream) {
  static std::atomic<bool> attr_set[kMaxDevices];
  const hb_status st = smem_limit_once(attr_set, ctx.device, chunk_e4m3_kernel<D, WIDEN>, TC<D, WIDEN>::SMEM,
                                       "cudaFuncSetAttribute(chunk_e4m3)");
  if (st != HB_OK) return st;
  return launch_pdl(chunk_e4m3_kernel<D, WIDEN>, grid, kThreads<WIDEN>, TC<D, WIDEN>::SMEM, stream,
                    "chunk_e4m3_kernel launch", tmQ, tmK, tmV, p);
}

template <int D>
hb_status launch_all(const DeviceCtx& ctx, const void* q, const Params& p, int grid, cudaStream_t stream) {
  CUtensorMap tmQ, tmK, tmV;
  hb_status st = encode_tmap_q3d(&tmQ, q, p.T, p.n_q, D);
  if (st != HB_OK) return st;
  const uint64_t rows = static_cast<uint64_t>(p.scratch_keys) * p.n_kv;
  st = encode_tmap_2d(&tmK, p.scratch_k, D, rows, D * 2, 64, TK, true);
  if (st != HB_OK) return st;
  st = encode_tmap_2d(&tmV, p.scratch_v, D, rows, D * 2, 64, TK, true);
  if (st != HB_OK) return st;
  st = launch_pdl(widen_kernel<D>, ctx.num_sms * 2, 256, 0, stream, "widen_kernel launch", p);
  if (st != HB_OK) return st;
  return launch_chunk<D, false>(ctx, tmQ, tmK, tmV, p, grid, stream);
}

template <int D>
hb_status launch_overflow(const DeviceCtx& ctx, const void* q, const Params& p, cudaStream_t stream) {
  CUtensorMap tmQ, tmK, tmV;
  hb_status st = encode_tmap_q3d(&tmQ, q, p.T, p.n_q, D);
  if (st != HB_OK) return st;
  // whole pages of codes, unswizzled: 16 rows of D bytes
  const uint64_t pool = static_cast<uint64_t>(p.num_pages) * p.n_kv * 16;
  st = encode_tmap_2d(&tmK, p.k, D, pool, D, D, 16, false, 1);
  if (st != HB_OK) return st;
  st = encode_tmap_2d(&tmV, p.v, D, pool, D, D, 16, false, 1);
  if (st != HB_OK) return st;
  return launch_chunk<D, true>(ctx, tmQ, tmK, tmV, p, ctx.num_sms, stream);
}

}  // namespace

hb_status chunk_e4m3_launch(const DeviceCtx& ctx, const void* q, const Params& p, int d_head, int grid,
                            cudaStream_t stream) {
  return d_head == 128 ? launch_all<128>(ctx, q, p, grid, stream) : launch_all<64>(ctx, q, p, grid, stream);
}

hb_status chunk_e4m3_overflow_launch(const DeviceCtx& ctx, const void* q, const Params& p, int d_head,
                                     cudaStream_t stream) {
  return d_head == 128 ? launch_overflow<128>(ctx, q, p, stream) : launch_overflow<64>(ctx, q, p, stream);
}

}  // namespace hb
