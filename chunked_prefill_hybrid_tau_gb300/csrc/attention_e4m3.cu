// Paged attention over a cache of E4M3 codes with a power-of-two scale per
// token and kv head (append_e4m3.cu).
//
//   out = sum_j P_j 2^ev_j V_j / sum_j P_j,  P_j = exp(2^ek_j (q . K_j) / sqrt(d) - m)
//
// Decode rows (sequences of one row): HBM bounds them, 2 n_kv (d + 1) bytes a
// key.  A unit is one row x one kv head x one range of kSplit keys at fixed
// positions, so a row's result does not depend on its batch; a warp owns whole
// units and streams their 16-token pages through a ring of its own, the next
// unit's pages behind the last ones without a pause.
//
// Both products run on m16n8k16 MMAs with the keys (S) or the head dimension
// (O) as rows and the kv head's q heads as the 8 columns:
//   S^T = K Q^T  : 16 keys x 8 heads, one MMA per 16 dims,
//   O^T += V^T P^T : 16 dims x 8 heads, one MMA per 16 dims of the output,
// half the MMAs and half the accumulators of the other way round.  More than 8
// q heads a kv head take a second column tile.  A 16-bit ldmatrix of 8-bit codes
// hands a lane four neighbouring dims of a key (K), or two dims of two keys (V,
// transposed); q's fragments follow the order that this gives the dims of S's
// sum, and O's rows 2 a and 2 a + 1 come to one lane.
//
// The codes are widened in registers, exactly.  K goes to fp16, for which there
// is an instruction (4 clocks a word of four codes; to bf16 it takes 10), and q
// with it: a q head is first multiplied by the power of two that takes its
// largest magnitude to 2^13, so that each of its values keeps its 8 bits unless
// it is below 2^-30 of the largest.  V stays bf16: its weights P 2^ev need
// the range.  2^ek multiplies the scores and 2^ev the weights, in fp32.
#include "attention_e4m3.cuh"

namespace hb {
namespace {

using namespace dev;
using namespace kv8;

// ---------------------------------------------------------------- decode rows
// 64 rows of 513 to 8189 keys, 8 kv heads of 128 (floor 86.1 us at the copy rate):
// 101 us back to back.  16 warps with 3 stages of 16 keys each: 12 with 4 103, 8
// with 6 128 (too few chains of conversions and MMAs in flight), 18 with 3 117 and
// 24 with 2 134 (fewer registers a thread); 20 with 2 as fast here, but one row of
// 32761 keys takes 26.4 us and not 24.1, 32 rows beside a chunk 61 and not 54.
// Units of 128 keys double the records, of 512 leave warps without one: both slower.
// All of it for up to 8 q heads a kv head; with 9 to 16 (two column tiles) the 128
// registers of 16 warps spill 304 bytes, and 64 such rows take 212 us (128 q heads on
// 8 of 128, floor 86.6).
constexpr int kSplit = 256;     // keys of a unit
constexpr int kDecWarps = 16;
constexpr float kRescale = 8.0f;  // log2 growth of a head's maximum that rescales its sums

// a split record: O [heads][D], the maximum and the sum of each head, fp32 (a multiple of 16 bytes)
__host__ __device__ constexpr int rec_floats(int grp, int d) { return grp * (d + 4); }

template <int D>
struct DC {
  static constexpr int PAGE = 16 * D;         // one page of one kv head, K or V
  static constexpr int STAGE = 2 * PAGE;
  static constexpr int DR = D == 128 ? 3 : 6;  // ring depth per warp
  static constexpr int OFF_SCALE = kDecWarps * DR * STAGE;  // K and V scales, 16 + 16 bytes a stage
  static constexpr int OFF_BAR = OFF_SCALE + kDecWarps * DR * 32;
  static constexpr int OFF_PRE = OFF_BAR + kDecWarps * DR * 8;
  static constexpr int SMEM = OFF_PRE + (kMaxSeqs + 1) * 4 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
};

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 8 x 8 matrix of 16-bit elements, transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Four codes as fp16, in their order.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Two codes of w as bf16: bytes 1 and 3, bytes 0 and 2.
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return mul_bf16x2(codes_moved(w), 0x7b807b80u); }
__device__ __forceinline__ uint32_t codes_even(uint32_t w) { return codes_odd(w << 8); }

// 2^e of a scale byte of the format: 27 .. 247, or 255 (NaN)
__device__ __forceinline__ float scale_of(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}
__device__ __forceinline__ uint2 ld_u2(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Byte offset of 16-byte piece c of key r in a swizzled page.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, int NT>
struct Heads {  // a warp's state of NT x 8 q heads
  uint32_t q[NT][D / 16][2];  // fp16, times a power of two
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2], f[NT][2];  // f: takes the sums of S to log2 units
};

// One 16-key page: S, the softmax step (a maximum that is raised only when it
// grows by more than 2^8, so that most pages need no reduction), O.  Lane (a =
// lane / 4, t = lane % 4) has keys a and a + 8 of heads 2 t and 2 t + 1.  `live`
// keys of the page count.
template <int D, int NT>
__device__ __forceinline__ void page_step(uint32_t kp, uint32_t vp, uint32_t sp, Heads<D, NT>& w, int live,
                                          int lane) {
  const int mat = lane >> 3, key = ((mat & 1) << 3) + (lane & 7), a = lane >> 2;
  float s[NT][4], s2[NT][4];  // two chains of dependent MMAs, not one
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
  for (int c = 0; c < D / 16; c += 2) {
    uint32_t r[4];
    ldsm_x4(kp + piece_at<D>(key, c + (mat >> 1)), r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t a0, a1, a2, a3;
      codes_f16(r[2 * i], a0, a2);
      codes_f16(r[2 * i + 1], a1, a3);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        mma16816<true>(i ? s2[n] : s[n], a0, a1, a2, a3, w.q[n][c + i][0], w.q[n][c + i][1]);
    }
  }
  const float k0 = scale_of(lds_u8(sp + a)), k1 = scale_of(lds_u8(sp + a + 8));
  const float v0 = scale_of(lds_u8(sp + 16 + a)), v1 = scale_of(lds_u8(sp + 16 + a + 8));
  const bool in0 = a < live, in1 = a + 8 < live;
  bool grew = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[n][h] = in0 ? (s[n][h] + s2[n][h]) * w.f[n][h] * k0 : -INFINITY;
      s[n][2 + h] = in1 ? (s[n][2 + h] + s2[n][2 + h]) * w.f[n][h] * k1 : -INFINITY;
      grew |= fmaxf(s[n][h], s[n][2 + h]) > w.m[n][h] + kRescale;
    }
  if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(s[n][h], s[n][2 + h]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        // per head: another head's growth must not move this one's maximum
        const float mn = mx > w.m[n][h] + kRescale ? mx : w.m[n][h];
        const float alpha = mn == w.m[n][h] ? 1.f : ex2_approx(w.m[n][h] - mn);
        w.m[n][h] = mn;
        w.l[n][h] *= alpha;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          w.o[n][i][h] *= alpha;
          w.o[n][i][2 + h] *= alpha;
        }
      }
  }
  uint32_t b[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float p[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float m = w.m[n][h] == -INFINITY ? 0.f : w.m[n][h];
      const float p0 = ex2_approx(s[n][h] - m), p1 = ex2_approx(s[n][2 + h] - m);
      w.l[n][h] += p0 + p1;
      p[h] = in0 ? p0 * v0 : 0.f;
      p[2 + h] = in1 ? p1 * v1 : 0.f;
    }
    b[n][0] = transpose8(pack_bf16x2(p[0], p[1]));
    b[n][1] = transpose8(pack_bf16x2(p[2], p[3]));
  }
#pragma unroll
  for (int c = 0; c < D / 16; c += 2) {
    uint32_t r[4];
    ldsm_x4_t(vp + piece_at<D>(key, c + (mat >> 1)), r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a0 = codes_even(r[2 * i]), a1 = codes_odd(r[2 * i]);
      const uint32_t a2 = codes_even(r[2 * i + 1]), a3 = codes_odd(r[2 * i + 1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816<false>(w.o[n][c + i], a0, a1, a2, a3, b[n][0], b[n][1]);
    }
  }
}

// The q heads of one row and kv head: fragments, empty sums.
template <int D, int NT>
__device__ __forceinline__ void take_heads(const Params& p, Heads<D, NT>& w, int row, int g, int lane) {
  const int a = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = 8 * n + a;
    const __nv_bfloat16* q = p.q + (static_cast<size_t>(row) * p.n_q + g * p.grp + (h < p.grp ? h : 0)) * D + 4 * t;
    uint32_t big = 0;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const uint2 v = ld_u2(q + 16 * c);
      w.q[n][c][0] = h < p.grp ? v.x : 0u;
      w.q[n][c][1] = h < p.grp ? v.y : 0u;
      big = max(big, max(v.x & 0x7fffu, (v.x >> 16) & 0x7fffu));
      big = max(big, max(v.y & 0x7fffu, (v.y >> 16) & 0x7fffu));
    }
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // 2^s takes the largest magnitude to 2^13; s at most 100, so that it and its
    // inverse are normal numbers
    const int s = min(13 + 127 - static_cast<int>(big >> 7), 100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - s) << 23) * p.scale_log2;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f = unpack_bf16x2(w.q[n][c][i]);
        const __half2 x = __floats2half2_rn(f.x * up, f.y * up);
        w.q[n][c][i] = *reinterpret_cast<const uint32_t*>(&x);
      }
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2) {
      w.f[n][h2] = __shfl_sync(0xffffffffu, down, (2 * t + h2) * 4);
      w.m[n][h2] = -INFINITY;
      w.l[n][h2] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) w.o[n][c][0] = w.o[n][c][1] = w.o[n][c][2] = w.o[n][c][3] = 0.f;
  }
}

// Units of every sequence before each one, into pre[0 .. S]: one-row sequences
// have n_kv per kSplit keys.  Lengths out of range are reported and have none.
__device__ __forceinline__ void count_units(const Params& p, int* pre) {
  for (int s = threadIdx.x; s < p.S; s += blockDim.x) {
    const int q0 = ld_s32(p.q_start + s), q1 = ld_s32(p.q_start + s + 1), kvl = ld_s32(p.kv_len + s);
    int n = 0;
    if (q0 < 0 || q1 > p.T || q1 <= q0 || kvl < q1 - q0 || kvl > p.max_kv_len || (kvl + 15) / 16 > p.max_pages ||
        (p.no_chunks && q1 - q0 != 1))
      flag_error(p.status, kStatusIndex);
    else if (q1 - q0 == 1)
      n = p.n_kv * ((kvl + kSplit - 1) / kSplit);
    pre[s + 1] = n;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    if (threadIdx.x == 0) pre[0] = 0;
    int carry = 0;
    for (int s0 = 0; s0 < p.S; s0 += 32) {
      const int s = s0 + static_cast<int>(threadIdx.x);
      int v = s < p.S ? pre[s + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (static_cast<int>(threadIdx.x) >= o) v += u;
      }
      if (s < p.S) pre[s + 1] = v + carry;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int upper_index(const int* pre, int n, int u) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int D, int NT>
__global__ void __launch_bounds__(kDecWarps * 32, 1)
    decode_e4m3_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Params p) {
  using C = DC<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* pre = reinterpret_cast<int*>(smem + C::OFF_PRE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * C::DR;
  uint8_t* ring = smem + warp * C::DR * C::STAGE;
  uint8_t* scales = smem + C::OFF_SCALE + warp * C::DR * 32;
  if (lane == 0) {
    for (int i = 0; i < C::DR; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (!p.wait_at_end) griddep_wait();
  griddep_launch_dependents();
  count_units(p, pre);
  const int total = pre[p.S];
  const int a = lane >> 2, t = lane & 3;
  // a unit: its sequence, kv head and split, its keys, and the ids of its pages
  // (lane b has that of page b)
  struct Work {
    int s, g, split, keys, whole, id;
  };
  auto look_up = [&](int u) {
    Work w = {0, 0, 0, 0, 0, 0};
    if (u < total) {
      w.s = upper_index(pre, p.S, u);
      const int local = u - pre[w.s];
      w.g = local % p.n_kv;
      w.split = local / p.n_kv;
      const int kvl = ld_s32(p.kv_len + w.s);
      w.keys = min(kvl - w.split * kSplit, kSplit);
      w.whole = kvl <= kSplit;
      if (lane * 16 < w.keys) {
        w.id = ld_s32(p.block_table + static_cast<size_t>(w.s) * p.max_pages + w.split * (kSplit / 16) + lane);
        if (w.id < 0 || w.id >= p.num_pages) {
          flag_error(p.status, kStatusIndex);
          w.id = 0;
        }
      }
    }
    return w;
  };
  int slot_in = 0, slot_out = 0;  // ring slots of the next copy and of the next page
  uint32_t phases = 0;            // bit s: parity to wait for on slot s
  auto issue = [&](const Work& w, int b) {
    const int at = (__shfl_sync(0xffffffffu, w.id, b) * p.n_kv + w.g) * 16;
    if (lane == 0) mbar_arrive_expect_tx(&full[slot_in], C::STAGE + 32);
    __syncwarp();
    // each byte is read once: first out of L2
    if (lane < 2)
      tma_load_2d_hint(ring + slot_in * C::STAGE + lane * C::PAGE, lane ? &tmV : &tmK, &full[slot_in], 0, at,
                       policy_evict_first());
    else if (lane < 4)
      bulk_load(scales + slot_in * 32 + (lane - 2) * 16, (lane == 2 ? p.ks : p.vs) + at, 16, &full[slot_in]);
    if (++slot_in == C::DR) slot_in = 0;
  };
  // neighbouring units on different SMs
  const int stride = kDecWarps * static_cast<int>(gridDim.x);
  int u = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  Work cur = look_up(u);
  int ahead = 0, flying = 0;  // pages of cur issued; pages of both on their way
  auto fill = [&](const Work& w, int& issued) {
    while (flying < C::DR && issued * 16 < w.keys) {
      issue(w, issued++);
      ++flying;
    }
  };
  fill(cur, ahead);
  bool ok = true;
  while (u < total && ok) {
    u += stride;
    const Work next = look_up(u);
    int early = 0;  // pages of next issued
    fill(next, early);
    const int row = ld_s32(p.q_start + cur.s);
    Heads<D, NT> w;
    take_heads<D, NT>(p, w, row, cur.g, lane);
    for (int b = 0; b * 16 < cur.keys; ++b) {
      const bool landed = mbar_wait(&full[slot_out], (phases >> slot_out) & 1u, nullptr, p.status);
      if (!__all_sync(0xffffffffu, landed)) {
        ok = false;
        break;
      }
      phases ^= 1u << slot_out;  // only now: the drain below waits for the phase that is still open
      const uint32_t kp = smem_u32(ring + slot_out * C::STAGE);
      page_step<D, NT>(kp, kp + C::PAGE, smem_u32(scales + slot_out * 32), w, cur.keys - 16 * b, lane);
      __syncwarp();
      if (++slot_out == C::DR) slot_out = 0;
      --flying;
      fill(cur, ahead);
      fill(next, early);
    }
    if (!ok) break;

    float* rec = p.partials +
                 ((static_cast<size_t>(cur.s) * p.max_splits + cur.split) * p.n_kv + cur.g) * rec_floats(p.grp, D);
    __nv_bfloat16* out = p.out + (static_cast<size_t>(row) * p.n_q + cur.g * p.grp) * D;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = w.l[n][h];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int head = 8 * n + 2 * t + h;
        if (head >= p.grp) continue;
        if (cur.whole) {
          const float inv = 1.f / l;
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            *reinterpret_cast<uint32_t*>(out + head * D + 16 * c + 2 * a) =
                pack_bf16x2(w.o[n][c][h] * inv, w.o[n][c][2 + h] * inv);
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            *reinterpret_cast<float2*>(rec + head * D + 16 * c + 2 * a) = make_float2(w.o[n][c][h], w.o[n][c][2 + h]);
          if (a == 0) {
            rec[p.grp * D + head] = w.m[n][h];
            rec[p.grp * (D + 1) + head] = l;
          }
        }
      }
    cur = next;
    ahead = early;
  }
  // after a wait that expired: the copies in flight land (bounded) before the warp leaves
  if (!ok && lane == 0)
    for (int i = 0; i < C::DR; ++i) mbar_drain(&full[i], (phases >> i) & 1u);
  if (p.wait_at_end) griddep_wait();
}

constexpr int kJoinWarps = 8, kJoin = 4;

// The parts of a chunk row whose keys are split (a CTA): a warp takes every
// eighth q head, all its records in flight.  The row's sequence is found ahead
// of the wait.
template <int D>
__device__ __forceinline__ void join_parts(const Params& p, int row, int warp, int lane) {
  constexpr int E = D / 32;
  int s = -1, q0 = 0, q1 = 0, kvl = 0;  // the last sequence that starts at or ahead of the row
  for (int i0 = 0; i0 < p.S; i0 += 32) {
    const bool ahead = i0 + lane < p.S && ld_s32(p.q_start + i0 + lane) <= row;
    s += __popc(__ballot_sync(0xffffffffu, ahead));
  }
  if (s >= 0) {
    q0 = ld_s32(p.q_start + s);
    q1 = ld_s32(p.q_start + s + 1);
    kvl = ld_s32(p.kv_len + s);
  }
  const int rows = q1 - q0;
  griddep_wait();  // by all: the kernel's end has to imply its predecessor's
  if (q0 < 0 || q1 > p.T || row < q0 || row >= q1 || (rows < 2 && !p.no_decodes) || kvl < rows ||
      kvl > p.max_kv_len || (kvl + 15) / 16 > p.max_pages)
    return;
  const int parts = part_count(p.n_q * ((rows + 127) / 128), first_tile_blocks(rows, kvl));
  if (parts == 1) return;
  for (int h = warp; h < p.n_q; h += kJoinWarps) {
    const float* rec = p.chunk_partials +
                       (static_cast<size_t>(part_row(p, row, s, q0)) * p.n_q + h) * p.max_parts * part_floats(D);
    float m[kMaxParts], l[kMaxParts], o[kMaxParts][E];
    float all = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) {
      // behind the last: the last again, with weight 0
      const float* at = rec + min(i, parts - 1) * part_floats(D);
      m[i] = ld_f32(at + D);
      l[i] = ld_f32(at + D + 1);
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = ld_f32(at + lane + 32 * e);
      all = fmaxf(all, m[i]);
    }
    if (all == -INFINITY) all = 0.f;
    float z = 0.f, x[E] = {};
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) {
      if (i >= parts) break;
      const float f = ex2_approx(m[i] - all);
      z += f * l[i];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] += f * o[i][e];
    }
    __nv_bfloat16* out = p.out + (static_cast<size_t>(row) * p.n_q + h) * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) out[32 * e] = __float2bfloat16_rn(x[e] / z);
  }
}

// The splits of one decode row and q head (a CTA), in an order of their number
// alone: warp w takes splits w, w + 8, ..., kJoin of them in flight with their
// maxima and sums; the warps' results are joined in order.  The plan is read
// ahead of the wait: the first kernel of the call (the widening, or the decode
// kernel) lets the next ones start only once everything ahead of it is complete.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_splits_kernel(Params p, int decode_items) {
  constexpr int E = D / 32;
  __shared__ float sum[kJoinWarps][D];
  __shared__ float2 state[kJoinWarps];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTAs of a decode row and q head, then of a chunk row
  const int item = static_cast<int>(blockIdx.x) - decode_items;
  if (item >= 0) {
    join_parts<D>(p, item, warp, lane);
    return;
  }
  const int s = blockIdx.x / p.n_q, h = blockIdx.x % p.n_q, g = h / p.grp, r = h % p.grp;
  const int q0 = ld_s32(p.q_start + s), q1 = ld_s32(p.q_start + s + 1), kvl = ld_s32(p.kv_len + s);
  griddep_wait();
  // as count_units: others were not computed, or were whole
  if (q0 < 0 || q1 > p.T || q1 - q0 != 1 || kvl <= kSplit || kvl > p.max_kv_len || (kvl + 15) / 16 > p.max_pages) return;
  const int n = (kvl + kSplit - 1) / kSplit;
  const size_t step = static_cast<size_t>(p.n_kv) * rec_floats(p.grp, D);
  const float* rec = p.partials + static_cast<size_t>(s) * p.max_splits * step +
                     static_cast<size_t>(g) * rec_floats(p.grp, D);
  float acc[E] = {}, l = 0.f, m = -INFINITY;
  for (int i0 = warp; i0 < n; i0 += kJoinWarps * kJoin) {
    float mi[kJoin], li[kJoin], o[kJoin][E];
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      // behind the last: the last again, with weight 0
      const int i = i0 + k * kJoinWarps;
      const float* at = rec + min(i, n - 1) * step;
      mi[k] = ld_f32(at + p.grp * D + r);
      li[k] = ld_f32(at + p.grp * (D + 1) + r);
      if (E == 4) {
        const float4 v = ld_f4(at + r * D + lane * E);
        o[k][0] = v.x, o[k][1] = v.y, o[k][2 % E] = v.z, o[k][3 % E] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) o[k][e] = ld_f32(at + r * D + lane * E + e);
      }
      if (i >= n) {
        mi[k] = -INFINITY;
        li[k] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[k][e] = 0.f;
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kJoin; ++k) mn = fmaxf(mn, mi[k]);
    const float mu = mn == -INFINITY ? 0.f : mn, alpha = ex2_approx(m - mu);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const float w = ex2_approx(mi[k] - mu);
      l += w * li[k];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w * o[k][e];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sum[warp][lane * E + e] = acc[e];
  if (lane == 0) state[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x < D / 2) {
    float all = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) all = fmaxf(all, state[w].x);
    if (all == -INFINITY) all = 0.f;
    float x = 0.f, y = 0.f, z = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = ex2_approx(state[w].x - all);
      x += f * sum[w][2 * threadIdx.x];
      y += f * sum[w][2 * threadIdx.x + 1];
      z += f * state[w].y;
    }
    *reinterpret_cast<uint32_t*>(p.out + (static_cast<size_t>(q0) * p.n_q + h) * D + 2 * threadIdx.x) =
        pack_bf16x2(x / z, y / z);
  }
}

template <int D, int NT>
hb_status decode_launch(const DeviceCtx& ctx, const CUtensorMap& tmK, const CUtensorMap& tmV, const Params& p, int grid,
                        cudaStream_t stream) {
  static std::atomic<bool> attr_set[kMaxDevices];
  const hb_status st = smem_limit_once(attr_set, ctx.device, decode_e4m3_kernel<D, NT>, DC<D>::SMEM,
                                       "cudaFuncSetAttribute(decode_e4m3)");
  if (st != HB_OK) return st;
  return launch_pdl(decode_e4m3_kernel<D, NT>, grid, kDecWarps * 32, DC<D>::SMEM, stream, "decode_e4m3_kernel launch",
                    tmK, tmV, p);
}

// SMs for the chunk kernel when both kinds of rows run side by side on
// disjoint SMs (each kernel's CTAs fill an SM's shared memory), from the plan's
// hints; 0: one after the other on all SMs.  It only moves work: no row's
// result depends on it.
//   chunk : units of a 128-row tile of a q head, kUnitUs and kBlockUs per 128
//           keys each, in rounds of n on n SMs;
//   decode: bytes at min(kDecodeBw, n kDecodeBwPerSm);
//   side by side: the longer, and kBeside of the shorter;
//   one after the other: both, and kTurnUs.
// Measured, 32 heads: 480 chunk rows behind 1024 keys beside 32 decodes 51.8 us
// on 43 SMs (as chosen) and one after the other, 55 on 64, 60 on 32; beside 8
// decodes 35.4 on 64 (as chosen), 38 one after the other; 2016 rows behind 4096
// keys beside 32 decodes 175 on 128 (as chosen), 181 one after the other.
constexpr double kUnitUs = 3.5;
constexpr double kBlockUs = 0.75;            // d_head 128
constexpr double kDecodeBwPerSm = 44000.0;   // bytes per us
constexpr double kDecodeBw = 6.0e6;
constexpr double kBeside = 0.12;
constexpr double kTurnUs = 7.0;

int chunk_sms(const DeviceCtx& ctx, const hb_device_plan& plan, const hb_layer_dims& dm) {
  const int S = ctx.num_sms;
  if (plan.chunk_pairs <= 0 || plan.decode_pairs <= 0 || plan.chunk_rows <= 0 || S < 4) return 0;
  const double dscale = dm.d_head / 128.0;
  // sequences of several rows, alike for want of more: the others have one each
  const double seqs = plan.n_seqs - (plan.n_rows - plan.chunk_rows) > 1
                          ? static_cast<double>(plan.n_seqs - (plan.n_rows - plan.chunk_rows)) : 1.0;
  double units = ceil(plan.chunk_rows / seqs / 128.0) * dm.n_q;
  double blocks = static_cast<double>(plan.chunk_pairs) / plan.chunk_rows / 128.0 + 0.5;
  const int parts = part_count(static_cast<int>(units < 1e6 ? units : 1e6),
                               static_cast<int>(blocks < 1e6 ? blocks : 1e6));
  units *= seqs * parts;
  blocks /= parts;
  const double t_unit = kUnitUs + blocks * kBlockUs * (0.5 + 0.5 * dscale);
  const double bytes = 2.0 * static_cast<double>(plan.decode_pairs) * dm.n_kv * (dm.d_head + 1);
  auto t_chunk = [&](int n) { return ceil(units / n) * t_unit; };
  auto t_decode = [&](int n) { return bytes / (n * kDecodeBwPerSm < kDecodeBw ? n * kDecodeBwPerSm : kDecodeBw); };
  int best = 0;
  double t_best = t_chunk(S) + t_decode(S) + kTurnUs;
  for (int n = 1; n < S; ++n) {
    const double tc = t_chunk(n), td = t_decode(S - n);
    const double t = tc > td ? tc + kBeside * td : td + kBeside * tc;
    if (t < t_best) {
      t_best = t;
      best = n;
    }
  }
  return best;
}

// Keys of several-row sequences that are widened ahead of the chunk kernel:
// what the sizes allow to come, but no more than this, and at least one
// sequence (1.07 GB with 8 kv heads of 128).
constexpr long long kScratchKeys = 262144;

long long chunk_keys(int rows, int seqs, int max_kv_len) {
  const long long n = seqs < rows / 2 ? seqs : rows / 2;
  return n * ((max_kv_len + 127ll) / 128 * 128);
}
long long scratch_keys(int rows, int seqs, int max_kv_len) {
  const long long all = chunk_keys(rows, seqs, max_kv_len), one = (max_kv_len + 127ll) / 128 * 128;
  const long long most = one > kScratchKeys ? one : kScratchKeys;
  return all < most ? all : most;
}

size_t partial_bytes(const hb_layer_dims& dm, int seqs, int max_kv_len) {
  const size_t splits = (static_cast<size_t>(max_kv_len) + kSplit - 1) / kSplit;
  const size_t recs = splits > 1 ? static_cast<size_t>(seqs) * splits * dm.n_kv : 0;
  return (recs * rec_floats(dm.n_q / dm.n_kv, dm.d_head) * 4 + 255) / 256 * 256;
}
// of chunk rows
int max_parts(const hb_layer_dims& dm, int max_kv_len) { return part_count(dm.n_q, (max_kv_len + 127ll) / 128); }
int part_stride(const hb_layer_dims& dm, int rows, int seqs) {
  return static_cast<long long>(seqs) * split_rows(dm.n_q) < rows ? split_rows(dm.n_q) : 0;
}
size_t chunk_partial_bytes(const hb_layer_dims& dm, int rows, int seqs, int max_kv_len) {
  const int parts = max_parts(dm, max_kv_len);
  const long long most = static_cast<long long>(seqs) * split_rows(dm.n_q);
  const size_t n = parts == 1 || rows < 2 ? 0 : most < rows ? most : rows;
  return (n * dm.n_q * parts * part_floats(dm.d_head) * 4 + 255) / 256 * 256;
}
size_t workspace_bytes(const hb_layer_dims& dm, int rows, int seqs, int max_kv_len) {
  const size_t scratch = static_cast<size_t>(scratch_keys(rows, seqs, max_kv_len)) * dm.n_kv * dm.d_head * 2;
  return 256 + partial_bytes(dm, seqs, max_kv_len) + chunk_partial_bytes(dm, rows, seqs, max_kv_len) + 2 * scratch;
}

}  // namespace
}  // namespace hb

extern "C" size_t hb_attention_e4m3_workspace_bytes(const hb_layer_dims* dims, int32_t max_rows, int32_t max_seqs,
                                                    int32_t max_kv_len) {
  if (!dims || max_rows < 0 || max_seqs < 0 || max_kv_len < 0 || dims->n_kv < 1 || dims->n_q < 1) return 0;
  return hb::workspace_bytes(*dims, max_rows, max_seqs, max_kv_len);
}

extern "C" hb_status hb_attention_e4m3(const void* q, const void* k_cache, const void* k_scale, const void* v_cache,
                                       const void* v_scale, int32_t num_pages, const hb_device_plan* plan,
                                       const hb_layer_dims* dims, int32_t max_kv_len, void* out, void* workspace,
                                       size_t ws_bytes, void* stream) {
  using namespace hb;
  clear_error();
  hb_status st = check_dims(dims);
  if (st != HB_OK) return st;
  HB_REQUIRE(plan != nullptr, "hb_attention_e4m3: null plan");
  HB_REQUIRE(plan->n_seqs >= 0 && plan->n_rows >= 0 && plan->max_pages >= 1, "hb_attention_e4m3: bad plan sizes");
  HB_REQUIRE(plan->n_seqs <= kMaxSeqs, "hb_attention_e4m3: at most %d sequences per iteration", kMaxSeqs);
  HB_REQUIRE(max_kv_len >= 1 && max_kv_len <= (1 << 28) && num_pages > 0,
             "hb_attention_e4m3: max_kv_len (at most 2^28) and num_pages must be positive");
  if (plan->n_seqs == 0 || plan->n_rows == 0) return HB_OK;
  HB_REQUIRE(q && k_cache && k_scale && v_cache && v_scale && out, "hb_attention_e4m3: null pointer");
  HB_REQUIRE(plan->seq_q_start && plan->seq_kv_len && plan->block_table, "hb_attention_e4m3: null plan array");
  HB_REQUIRE(plan->n_rows >= plan->n_seqs, "hb_attention_e4m3: every sequence has at least one row (%d rows, %d sequences)",
             plan->n_rows, plan->n_seqs);
  HB_REQUIRE(aligned16(q) && aligned16(out) && aligned16(k_cache) && aligned16(v_cache) && aligned16(k_scale) &&
                 aligned16(v_scale),
             "hb_attention_e4m3: 16-byte alignment");
  const bool no_chunks = plan->n_rows == plan->n_seqs;
  const size_t need = workspace_bytes(*dims, no_chunks ? 0 : plan->n_rows, plan->n_seqs, max_kv_len);
  HB_REQUIRE(workspace != nullptr && ws_bytes >= need, "hb_attention_e4m3: workspace of %zu bytes needed, %zu given",
             need, ws_bytes);
  HB_REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0,
             "hb_attention_e4m3: workspace must be 256-byte aligned");
  DeviceCtx ctx;
  st = device_context(&ctx);
  if (st != HB_OK) return st;
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.k = static_cast<const uint8_t*>(k_cache);
  p.ks = static_cast<const uint8_t*>(k_scale);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.vs = static_cast<const uint8_t*>(v_scale);
  p.q_start = plan->seq_q_start;
  p.kv_len = plan->seq_kv_len;
  p.block_table = plan->block_table;
  p.S = plan->n_seqs;
  p.T = plan->n_rows;
  p.max_pages = plan->max_pages;
  p.num_pages = num_pages;
  p.n_q = dims->n_q;
  p.n_kv = dims->n_kv;
  p.grp = dims->n_q / dims->n_kv;
  p.max_kv_len = max_kv_len;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(dims->d_head)));
  p.status = ctx.status;
  p.partials = static_cast<float*>(workspace);
  p.scratch_keys = no_chunks ? 0 : static_cast<int>(scratch_keys(plan->n_rows, plan->n_seqs, max_kv_len));
  uint8_t* at = static_cast<uint8_t*>(workspace) + partial_bytes(*dims, plan->n_seqs, max_kv_len);
  p.chunk_partials = reinterpret_cast<float*>(at);
  p.part_stride = part_stride(*dims, plan->n_rows, plan->n_seqs);
  p.max_parts = max_parts(*dims, max_kv_len);
  at += chunk_partial_bytes(*dims, no_chunks ? 0 : plan->n_rows, plan->n_seqs, max_kv_len);
  p.scratch_k = reinterpret_cast<__nv_bfloat16*>(at);
  p.scratch_v = p.scratch_k + static_cast<size_t>(p.scratch_keys) * dims->n_kv * dims->d_head;
  p.max_splits = (max_kv_len + kSplit - 1) / kSplit;
  p.no_chunks = no_chunks;
  p.no_decodes = plan->n_seqs == 1 && plan->n_rows > 1;
  p.wait_at_end = 0;
  const uint64_t rows = static_cast<uint64_t>(num_pages) * dims->n_kv * 16;
  HB_REQUIRE(rows <= INT32_MAX, "hb_attention_e4m3: num_pages * n_kv * 16 must be below 2^31");
  HB_REQUIRE(static_cast<int64_t>(p.scratch_keys) * dims->n_kv <= INT32_MAX,
             "hb_attention_e4m3: max_kv_len * n_kv must be below 2^31");
  CUtensorMap tmK, tmV;
  st = encode_tmap_code_pages(&tmK, k_cache, rows, dims->d_head);
  if (st != HB_OK) return st;
  st = encode_tmap_code_pages(&tmV, v_cache, rows, dims->d_head);
  if (st != HB_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = ctx.num_sms;  // of the decode kernel
  if (!p.no_chunks) {
    const int nc = p.no_decodes ? 0 : chunk_sms(ctx, *plan, *dims);
    st = chunk_e4m3_launch(ctx, q, p, dims->d_head, nc > 0 ? nc : ctx.num_sms, s);
    if (st != HB_OK) return st;
    sms -= nc;
    p.wait_at_end = 1;
  }
  if (p.no_decodes)
    st = HB_OK;
  else if (dims->d_head == 128)
    st = p.grp <= 8 ? decode_launch<128, 1>(ctx, tmK, tmV, p, sms, s) : decode_launch<128, 2>(ctx, tmK, tmV, p, sms, s);
  else
    st = p.grp <= 8 ? decode_launch<64, 1>(ctx, tmK, tmV, p, sms, s) : decode_launch<64, 2>(ctx, tmK, tmV, p, sms, s);
  // behind the decode kernel, which runs beside the first: most calls that may
  // have such sequences have none (32 decodes and a chunk with a max_kv_len of 32768
  // take 56 us, with their own maximum, 4097, 50)
  if (st == HB_OK && !p.no_chunks && chunk_keys(p.T, p.S, max_kv_len) > p.scratch_keys)
    st = chunk_e4m3_overflow_launch(ctx, q, p, dims->d_head, s);
  const int decode_items = p.no_decodes || p.max_splits == 1 ? 0 : p.S * p.n_q;
  const int items = decode_items + (p.no_chunks || p.max_parts == 1 ? 0 : p.T);
  if (st != HB_OK || items == 0) return st;
  return launch_pdl(dims->d_head == 128 ? join_splits_kernel<128> : join_splits_kernel<64>, items,
                    kJoinWarps * 32, 0, s, "join_splits_kernel launch", p, decode_items);
}
