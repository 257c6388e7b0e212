// Attention of prompt chunks over a cache of E4M3 codes, on the
// 5th-generation tensor cores.
//
// A chunk's query at position p attends to keys 0..p of its request
// (Sarathi-Serve reading notes, sections 3.1 and 7.5b):
//   S = Q K^T, P = 2^(S scale - m), O += P V, out = O / sum P,
// K = 2^ek codes and V = 2^ev codes widened to bf16, which is exact (powers of
// two), so the products are those of hb_attention with such a cache in bf16.
//
// Unit: two 128-row tiles of one kv head -- (row tile, q head) pairs in that
// order, so with an even number of q heads per kv head two heads of the same
// rows -- and keys 0 .. last in blocks of 128.  Both tiles use every widened
// block, which halves the widening a tile pays for; codes are half the bytes
// that bf16 pages would bring in.
//
// Warp roles (448 threads, one CTA per SM):
//   warp 0      finds the unit (its lanes scan the sequences), publishes it in
//               shared memory, loads both Q tiles and, 64 keys a slot, the
//               block's K and V codes with their scale bytes into a ring;
//   warps 10-13 widen: a warp takes one 16-key page of a slot, 16 codes a lane
//               at a time, into the 128-byte swizzled K or V block; keys behind
//               the unit's last become zeros;
//   warp 1      MMA issuer (one thread): S_x = Q_x K_j^T (M = N = 128) into
//               tile x's tensor-memory columns, O_x += P_x V_j with P_x read
//               from the same columns (bf16, written over S_x), whichever has
//               its inputs; while one tile's softmax runs, the other's MMAs do;
//   warps 2-5, 6-9  softmax of tile 0 and 1: a thread has one row, reads S once
//               for the maximum and once more for the exponentials, 32 columns
//               at a time; O is rescaled only where a row's maximum grew by
//               more than 2^8; at the end O / l to global memory.
// A value whose scale is NaN must reach the rows that see its key and no other:
// 0 * NaN would spread it, so the widening puts the NaN into the key's K row
// (S is masked by selection) and zeros into V.
// Every wait is bounded; an expired wait sets the status word and unwinds.
#include "attention_e4m3.cuh"
#include "attention_tc.cuh"

namespace hb {
namespace {

using namespace dev;
using kv8::mul_bf16x2;
using kv8::Params;
using tc::mma_bf16_ts;
using tc::smem_desc_sw128_mn;
using tc::tmem_st_32x32b_x32;
using tc::tmem_st_wait;

constexpr int TQ = 128, TK = 128;
constexpr int HK = 64;  // keys of a ring slot
constexpr int kStages = 2;
constexpr int kSoft0 = 2, kConv0 = 10, kConvWarps = 4;
constexpr int kThreads = 32 * (kConv0 + kConvWarps);
constexpr float kRescale = 8.0f;

struct Tile {
  int row0, nrows, pos0, head;  // nrows 0: the unit has one tile
};
struct Unit {
  int valid, seq, g, nblk;
  Tile t[2];
};

template <int D>
struct TC {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_TILE = 128 * 128;        // 128 rows x 128 bytes (64 dims)
  static constexpr int TILE = HALVES * HALF_TILE;    // a Q tile, a K or V block
  static constexpr int SLOTS = D == 128 ? 4 : 8;
  static constexpr int SLOT = HK * D;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + kStages * TILE;
  static constexpr int OFF_C = OFF_V + kStages * TILE;
  static constexpr int OFF_S = OFF_C + SLOTS * SLOT;  // scales: K's (or V's) 64 bytes, V's 64 bytes beside K
  static constexpr int OFF_U = OFF_S + SLOTS * 2 * HK;
  static constexpr int OFF_BAR = OFF_U + 2 * 64;
  static constexpr int SMEM = OFF_BAR + 400 + 1024;
  static_assert(sizeof(Unit) <= 64 && SMEM <= 232448, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;  // S0 S1 (P over them) O0 O1
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

// The tile that is the i-th of its kv head, heaviest rows first.
__device__ __forceinline__ Tile tile_of(const Params& p, int i, int ntiles, int g, int q0, int qlen, int kvl) {
  Tile t = {0, 0, 0, 0};
  if (i < ntiles * p.grp) {
    const int rt = ntiles - 1 - i / p.grp;
    t.head = g * p.grp + i % p.grp;
    t.row0 = q0 + rt * TQ;
    t.nrows = min(TQ, qlen - rt * TQ);
    t.pos0 = kvl - qlen + rt * TQ;
  }
  return t;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_e4m3_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, Params p) {
  using C = TC<D>;
  // the decode kernel behind this one starts beside it once its inputs are there
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sC = smem + C::OFF_C;
  uint8_t* sS = smem + C::OFF_S;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* u_full = bar;            // [2] unit published
  uint64_t* u_empty = bar + 2;       // [2] MMA warp, softmax warps, widening warps have read it
  uint64_t* q_full = bar + 4;
  uint64_t* q_empty = bar + 5;
  uint64_t* c_full = bar + 6;        // [SLOTS] codes and scales landed
  uint64_t* c_empty = bar + 14;      // [SLOTS] widening warps
  uint64_t* k_full = bar + 22;       // [2] widening warps
  uint64_t* k_empty = bar + 24;      // [2]
  uint64_t* v_full = bar + 26;
  uint64_t* v_empty = bar + 28;
  uint64_t* s_full = bar + 30;       // [2] by tile
  uint64_t* p_full = bar + 32;       // [2] four softmax warps
  uint64_t* pv_done = bar + 34;      // [2]
  uint64_t* o_empty = bar + 36;      // [2] four softmax warps
  uint64_t* drain = bar + 38;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 39);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Unit* units = reinterpret_cast<Unit*>(smem + C::OFF_U);  // [2], 64 bytes apart

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], 1 + 8 + kConvWarps);
      mbar_init(&k_full[i], kConvWarps);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], kConvWarps);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_empty[i], 4);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], kConvWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
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
    w = *reinterpret_cast<const Unit*>(reinterpret_cast<const uint8_t*>(units) + (n & 1) * 64);
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[n & 1]);
    return w.valid != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    int s0 = 0, before = 0;  // units of the sequences ahead of s0
    int slot = 0;
    uint32_t cph = 0, pending = 0, armed = 0;
    bool ok = true;
    for (int n = 0, v = blockIdx.x; ok; ++n, v += gridDim.x) {
      // the sequence that unit v falls into, 32 at a time
      Unit w;
      w.valid = 0;
      while (s0 < p.S && !w.valid) {
        const int s = s0 + lane;
        int count = 0, q0 = 0, qlen = 0, kvl = 0;
        if (s < p.S) {
          q0 = ld_s32(p.q_start + s);
          const int q1 = ld_s32(p.q_start + s + 1);
          qlen = q1 - q0;
          kvl = ld_s32(p.kv_len + s);
          if (q0 < 0 || q1 > p.T || qlen < 1 || kvl < qlen || kvl > p.max_kv_len || (kvl + 15) / 16 > p.max_pages ||
              (p.no_decodes && qlen < 2))
            flag_error(p.status, kStatusIndex);
          else if (qlen > 1)
            count = p.n_kv * (((qlen + TQ - 1) / TQ * p.grp + 1) / 2);
        }
        int upto = count;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int u = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += u;
        }
        upto += before;
        const unsigned mine = __ballot_sync(0xffffffffu, v < upto);
        if (mine == 0) {
          before = __shfl_sync(0xffffffffu, upto, 31);
          s0 += 32;
          continue;
        }
        const int at = __ffs(static_cast<int>(mine)) - 1;
        const int local = v - __shfl_sync(0xffffffffu, upto - count, at);
        q0 = __shfl_sync(0xffffffffu, q0, at);
        qlen = __shfl_sync(0xffffffffu, qlen, at);
        kvl = __shfl_sync(0xffffffffu, kvl, at);
        const int ntiles = (qlen + TQ - 1) / TQ;
        w.valid = 1;
        w.seq = s0 + at;
        w.g = local % p.n_kv;
        const int i = local / p.n_kv * 2;
        w.t[0] = tile_of(p, i, ntiles, w.g, q0, qlen, kvl);
        w.t[1] = tile_of(p, i + 1, ntiles, w.g, q0, qlen, kvl);
        // the second tile's rows are the same or earlier ones
        w.nblk = (w.t[0].pos0 + w.t[0].nrows + TK - 1) / TK;
      }
      if (lane == 0) {
        ok = mbar_wait(&u_empty[n & 1], ((n >> 1) & 1) ^ 1u, abort_flag, p.status);
        if (ok) {
          *reinterpret_cast<Unit*>(reinterpret_cast<uint8_t*>(units) + (n & 1) * 64) = w;
          mbar_arrive(&u_full[n & 1]);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) ok = false;
      if (!ok || !w.valid) break;
      const int tiles = w.t[1].nrows ? 2 : 1;
      if (lane == 0) {
        ok = mbar_wait(q_empty, (n & 1) ^ 1u, abort_flag, p.status);
        if (ok) {
          mbar_arrive_expect_tx(q_full, tiles * C::TILE);
          for (int x = 0; x < tiles; ++x)
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf)
              tma_load_3d(sQ + x * C::TILE + hf * C::HALF_TILE, &tmQ, q_full, hf * 64, w.t[x].head, w.t[x].row0);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) {
        ok = false;
        break;
      }
      const int* bt = p.block_table + static_cast<size_t>(w.seq) * p.max_pages;
      const int key_end = w.t[0].pos0 + w.t[0].nrows;
      const int npages = (key_end + 15) / 16;
      // lane l < 8 has the id of page l of a block, loaded two blocks ahead
      auto load_page = [&](int j) { return lane < 8 && j * 8 + lane < npages ? ld_s32(bt + j * 8 + lane) : 0; };
      int pf0 = load_page(0), pf1 = load_page(1);
      for (int j = 0; j < w.nblk && ok; ++j) {
        int cur = pf0;
        pf0 = pf1;
        pf1 = load_page(j + 2);
        if (cur < 0 || cur >= p.num_pages) {
          flag_error(p.status, kStatusIndex);
          cur = 0;
        }
#pragma unroll 1
        for (int i = 0; i < 4 && ok; ++i) {  // K keys 0..63, 64..127, V the same
          const bool is_v = i >= 2;
          const int pg = (i & 1) * 4;
          const int here = max(0, min(4, npages - j * 8 - pg));
          if (lane == 0) {
            ok = mbar_wait(&c_empty[slot], cph ^ 1u, abort_flag, p.status);
            if (ok) {
              pending |= 1u << slot;
              armed = (armed & ~(1u << slot)) | (cph << slot);
              mbar_arrive_expect_tx(&c_full[slot], here * (16 * D + (is_v ? 16 : 32)));
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          // lanes 0..3 a page of codes each, 4..7 its scales, 8..11 V's beside K's
          const int l4 = lane & 3;
          const int at = (__shfl_sync(0xffffffffu, cur, pg + l4) * p.n_kv + w.g) * 16;
          if (ok && lane < 12 && l4 < here) {
            if (lane < 4)
              tma_load_2d(sC + slot * C::SLOT + l4 * 16 * D, is_v ? &tmV : &tmK, &c_full[slot], 0, at);
            else if (lane < 8)
              bulk_load(sS + slot * 2 * HK + l4 * 16, (is_v ? p.vs : p.ks) + at, 16, &c_full[slot]);
            else if (!is_v)
              bulk_load(sS + slot * 2 * HK + HK + l4 * 16, p.vs + at, 16, &c_full[slot]);
          }
          if (++slot == C::SLOTS) {
            slot = 0;
            cph ^= 1u;
          }
        }
      }
    }
    if (!ok && lane == 0)
      for (int s = 0; s < C::SLOTS; ++s)
        if (pending & (1u << s)) mbar_drain(&c_full[s], (armed >> s) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = lane == 0;
    constexpr uint32_t idS = idesc_bf16_f32(TQ, TK);
    constexpr uint32_t idPV = idesc_bf16_f32(TQ, D) | (1u << 16);  // B (V) is MN-major
    int J = 0;                // blocks of the units before
    int nS[2] = {0, 0};       // S and PV blocks of each tile in the units before
    int nU[2] = {0, 0};       // units of each tile
    bool ok = true;
    Unit w;
    for (int n = 0; ok && next_unit(n, w); ++n) {
      if (leader) {
        const int tiles = w.t[1].nrows ? 2 : 1;
        ok = mbar_wait(q_full, n & 1, abort_flag, p.status);
        int js[2] = {0, 0}, jp[2] = {0, 0};
        if (tiles == 1) js[1] = jp[1] = w.nblk;
        bool o_free[2] = {false, false};
        uint64_t t0 = globaltimer();
        while (ok && (jp[0] < w.nblk || jp[1] < w.nblk)) {
          bool progressed = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (jp[x] < js[x]) {
              const int gv = J + jp[x], st = gv % kStages, use = nS[x] + jp[x];
              if (!o_free[x]) o_free[x] = mbar_test(&o_empty[x], (nU[x] & 1) ^ 1u);
              if (o_free[x] && mbar_test(&p_full[x], use & 1) && mbar_test(&v_full[st], (gv / kStages) & 1)) {
                tc_fence_after();
                const uint32_t v_addr = smem_u32(sV + st * C::TILE);
#pragma unroll
                for (int kk = 0; kk < TK / 16; ++kk)
                  mma_bf16_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8,
                              smem_desc_sw128_mn(v_addr + kk * 2048, C::HALF_TILE, 1024), idPV,
                              (jp[x] > 0 || kk > 0) ? 1u : 0u);
                ++jp[x];
                if (jp[x ^ 1] >= jp[x]) mma_commit(&v_empty[st]);  // both tiles have used the block
                mma_commit(&pv_done[x]);
                progressed = true;
              }
            }
            // S_x is written over P_x: its PV has to be complete
            if (js[x] < w.nblk && js[x] == jp[x]) {
              const int gk = J + js[x], st = gk % kStages, use = nS[x] + js[x];
              if (mbar_test(&pv_done[x], (use & 1) ^ 1u) && mbar_test(&k_full[st], (gk / kStages) & 1)) {
                tc_fence_after();
                const uint32_t q_addr = smem_u32(sQ + x * C::TILE), k_addr = smem_u32(sK + st * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t off = (kk >> 2) * C::HALF_TILE + (kk & 3) * 32;
                  mma_bf16(tmem + x * 128, smem_desc_sw128(q_addr + off), smem_desc_sw128(k_addr + off), idS,
                           kk > 0 ? 1u : 0u);
                }
                ++js[x];
                if (js[x ^ 1] >= js[x]) {
                  mma_commit(&k_empty[st]);
                  if (js[x] == w.nblk) mma_commit(q_empty);
                }
                mma_commit(&s_full[x]);
                progressed = true;
              }
            }
          }
          if (progressed) {
            t0 = globaltimer();
          } else if (*abort_flag) {
            ok = false;
          } else if (globaltimer() - t0 > kWaitTimeoutNs) {
            flag_error(p.status, kStatusTimeout);
            *abort_flag = 1;
            ok = false;
          }
        }
        J += w.nblk;
        for (int x = 0; x < tiles; ++x) {
          nS[x] += w.nblk;
          ++nU[x];
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    if (leader && !ok) {
      // nothing may still read shared memory or write tensor memory at the end
      mma_commit(drain);
      mbar_drain(drain, 0);
    }
  } else if (warp >= kConv0) {
    // ------------------------------------------------------------ widening
    const int cw = warp - kConv0;  // page of a slot
    constexpr int PIECES = D / 16;  // 16-code pieces of a key
    const int c = lane % PIECES;
    int slot = 0, J = 0;
    uint32_t cph = 0;
    bool ok = true;
    Unit w;
    for (int n = 0; ok && next_unit(n, w); ++n) {
      const int key_end = w.t[0].pos0 + w.t[0].nrows;
      for (int j = 0; j < w.nblk && ok; ++j) {
        const int st = (J + j) % kStages, use = (J + j) / kStages;
#pragma unroll 1
        for (int kv = 0; kv < 2 && ok; ++kv) {
          uint8_t* dst = (kv ? sV : sK) + st * C::TILE;
          bool free = mbar_wait(kv ? &v_empty[st] : &k_empty[st], (use & 1) ^ 1u, abort_flag, p.status);
          if (!__all_sync(0xffffffffu, free)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            bool landed = mbar_wait(&c_full[slot], cph, abort_flag, p.status);
            if (!__all_sync(0xffffffffu, landed)) {
              ok = false;
              break;
            }
            const uint8_t* codes = sC + slot * C::SLOT + cw * 16 * D;
            const uint8_t* scales = sS + slot * 2 * HK + cw * 16;
            constexpr int STEPS = 16 * PIECES / 32;  // 16-code pieces of a lane
            uint4 raw[STEPS];
            uint32_t sb[STEPS];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
              const int r = i * (32 / PIECES) + lane / PIECES;
              raw[i] = *reinterpret_cast<const uint4*>(codes + r * D + c * 16);
              sb[i] = scales[r];
              // a NaN value goes into its key
              if (kv == 0 && scales[HK + r] == 255) sb[i] = 255;
              if (kv == 1 && sb[i] == 255) sb[i] = 256;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_empty[slot]);
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
              const int r = hf * HK + cw * 16 + i * (32 / PIECES) + lane / PIECES;  // key of the block
              Factor f = factor_of(sb[i]);
              if (j * TK + r >= key_end || sb[i] == 256) f.first = 0, f.second = 0x3f803f80u;
              const uint32_t word[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[2 * e] = mul_bf16x2(kv8::codes_moved(__byte_perm(word[e], 0, 0x1404)), f.first);
                o[2 * e + 1] = mul_bf16x2(kv8::codes_moved(__byte_perm(word[e], 0, 0x3424)), f.first);
              }
              if (__any_sync(0xffffffffu, f.second != 0x3f803f80u)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(o[e], f.second);
              }
              // 16 dims: two 16-byte chunks of row r in their 64-dim half.  Lanes of
              // the upper half store theirs in the other order: the eight lanes of
              // a key then meet eight different banks
              const int flip = c >> 2;
              uint8_t* row = dst + (c >> 2) * C::HALF_TILE + r * 128;
              const int j0 = 2 * (c & 3);
              const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
              *reinterpret_cast<uint4*>(row + (((j0 + flip) ^ (r & 7)) << 4)) = flip ? hi : lo;
              *reinterpret_cast<uint4*>(row + (((j0 + (flip ^ 1)) ^ (r & 7)) << 4)) = flip ? lo : hi;
            }
            if (++slot == C::SLOTS) {
              slot = 0;
              cph ^= 1u;
            }
          }
          if (!ok) break;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv ? &v_full[st] : &k_full[st]);
        }
      }
      J += w.nblk;
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int x = (warp - kSoft0) >> 2;  // tile
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t tS = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + x * 128;
    const uint32_t tO = tS + 256;
    int use = 0;
    Unit w;
    for (int n = 0; next_unit(n, w); ++n) {
      const Tile t = w.t[x];
      if (t.nrows == 0) continue;
      const int lim = r < t.nrows ? t.pos0 + r : t.pos0 + t.nrows - 1;  // last key this row sees
      float m_used = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < w.nblk; ++j, ++use) {
        bool sok = mbar_wait(&s_full[x], use & 1, abort_flag, p.status);
        if (!__all_sync(0xffffffffu, sok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int seen = lim - j * TK;  // columns 0 .. seen of the block
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < TK; c += 64) {
          uint32_t sv[64];
          tmem_ld_32x32b_x32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld_32x32b_x32(tS + c + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          tmem_ld_wait();
          if (seen >= c + 63) {
#pragma unroll
            for (int e = 0; e < 64; ++e) mx = fmaxf(mx, __uint_as_float(sv[e]));
          } else {
#pragma unroll
            for (int e = 0; e < 64; ++e) mx = fmaxf(mx, c + e <= seen ? __uint_as_float(sv[e]) : -INFINITY);
          }
        }
        mx *= p.scale_log2;
        const bool raise = mx > m_used + kRescale;
        const float m_new = raise ? mx : m_used;
        const float alpha = raise ? ex2_approx(m_used - m_new) : 1.f;
        // S of this block was issued behind the PV of the last one: O is complete
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t ov[32];
            tmem_ld_32x32b_x32(tO + c, ov);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st_32x32b_x32(tO + c, ov);
          }
        }
        m_used = m_new;
        l *= alpha;
        const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
        float rs = 0.f;
#pragma unroll
        for (int c = 0; c < TK; c += 64) {
          uint32_t sv[64], pk[32];
          tmem_ld_32x32b_x32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld_32x32b_x32(tS + c + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          tmem_ld_wait();
          if (seen < c + 63) {
#pragma unroll
            for (int e = 0; e < 64; ++e) sv[e] = c + e <= seen ? sv[e] : 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float a0 = ex2_approx(fmaf(__uint_as_float(sv[2 * e]), p.scale_log2, neg_m));
            const float a1 = ex2_approx(fmaf(__uint_as_float(sv[2 * e + 1]), p.scale_log2, neg_m));
            rs += a0 + a1;
            pk[e] = pack_bf16x2(a0, a1);
          }
          // over columns of S that are in registers already
          tmem_st_32x32b_x32(tS + c / 2, pk);
        }
        l += rs;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      bool pok = mbar_wait(&pv_done[x], (use - 1) & 1, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, pok)) break;
      tc_fence_after();
      const float inv = 1.f / l;
      __nv_bfloat16* orow = p.out + (static_cast<size_t>(t.row0 + r) * p.n_q + t.head) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t ov[32];
        tmem_ld_32x32b_x32(tO + c, ov);
        tmem_ld_wait();
        if (r < t.nrows) {
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
      if (lane == 0) mbar_arrive(&o_empty[x]);  // O was read into registers
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D>
hb_status launch_chunk(const DeviceCtx& ctx, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                       const Params& p, int grid, cudaStream_t stream) {
  static std::atomic<bool> attr_set[kMaxDevices];
  const hb_status st =
      smem_limit_once(attr_set, ctx.device, chunk_e4m3_kernel<D>, TC<D>::SMEM, "cudaFuncSetAttribute(chunk_e4m3)");
  if (st != HB_OK) return st;
  return launch_pdl(chunk_e4m3_kernel<D>, grid, kThreads, TC<D>::SMEM, stream, "chunk_e4m3_kernel launch", tmQ, tmK, tmV,
                    p);
}

}  // namespace

hb_status chunk_e4m3_launch(const DeviceCtx& ctx, const void* q, const void* k_cache, const void* v_cache,
                            const kv8::Params& p, int d_head, int grid, cudaStream_t stream) {
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t rows = static_cast<uint64_t>(p.num_pages) * p.n_kv * 16;
  hb_status st = encode_tmap_q3d(&tmQ, q, p.T, p.n_q, d_head);
  if (st != HB_OK) return st;
  // whole pages of codes, unswizzled: 16 rows of d_head bytes
  st = encode_tmap_2d(&tmK, k_cache, d_head, rows, d_head, d_head, 16, false, 1);
  if (st != HB_OK) return st;
  st = encode_tmap_2d(&tmV, v_cache, d_head, rows, d_head, d_head, 16, false, 1);
  if (st != HB_OK) return st;
  return d_head == 128 ? launch_chunk<128>(ctx, tmQ, tmK, tmV, p, grid, stream)
                       : launch_chunk<64>(ctx, tmQ, tmK, tmV, p, grid, stream);
}

}  // namespace hb
