// Log probabilities of given tokens, the entropy and the k best alternatives
// of every row of logits, in one read of the logits.
//
// With m = max x_i, s = sum exp(x_i - m), t = sum exp(x_i - m) (x_i - m):
//   lse = m + log s,  log p_i = (x_i - m) - log s,  entropy = log s - t / s,
// so one pass that carries (m, s, t) has everything but the order; two parts
// of a row join by rescaling to the larger m.  The differences x - m are
// formed before the product with log2(e): rounding m log2(e) first would put
// an error of m * 2^-24 into every term.
//
// The k best: every thread keeps the largest of its elements.  Four lanes'
// largest make a group; of the CTA's 64 groups the k-th largest is a bound that
// at least k elements reach, and only threads whose largest reaches it (k, and
// some more) can hold one of the k best.  Their elements are read again (a 256th
// of the row each, from L2), those at or above the bound are collected (a few
// more than k) and ranked by counting.
//
// A row has 8 fixed segments, and thread t of a segment fixed elements; states
// join over segments first, in a fixed tree, then over threads.  1, 2, 4 or 8
// CTAs (a cluster) share a row's segments, more the fewer rows there are: the
// arithmetic, and so every bit, is the same.
//
// Reads 4 or 2 bytes an element once: HBM bounds it for many rows, 2048 x 64000
// bf16 in 59 us (floor 39.2 at the copy rate).  52 of these are the pass itself:
// the issue slots are 79% busy, 13 instructions an element, and a CTA that starts,
// ends or joins has no loads in flight, which four CTAs of 64 registers cover only
// in part (five spill); the 8 best cost 7 us, 32 cost 22.
// 2048 x 32000 fp32: 54 us, 700 rows 19 (floor 13.4).  Where fewer than k groups hold
// a finite logit (a mask that leaves a few tokens; vocabularies of a few thousand) the
// bound is -inf and the row is read again for exact keys: 64 x 32000 fp32 with 12
// tokens left 144 us, unmasked 12.7.
// One row takes 7 us, most of it in the cluster's barriers and the chain of the
// selection.
#include <cuda_bf16.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSegs = 8;
constexpr int P = 4;                  // 16-byte pieces that a thread takes at a time
constexpr int kGroups = kThreads / 4;
constexpr int kMaxTop = 32;
constexpr int kCap = 1024;            // collected candidates
constexpr float kLeast = -1e30f;      // stands for differences of -infinity, where the factor is 0
constexpr float kLog2e = 1.44269504088896341f;

struct Args {
  const void* logits;
  long long stride;
  int vocab;
  const int* tokens;
  int n_tokens;
  float* token_lp;
  float* entropy;
  int top_k;
  int* top_ids;
  float* top_lp;
  int* status;
};

struct State {
  float m, s, t;
};
struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
};

// The states of two parts of a row as one.
__device__ __forceinline__ State join(const State& a, const State& b) {
  const float m = fmaxf(a.m, b.m);
  // a part without a finite logit, or an empty one, has m = -inf and s = 0
  // (and a difference that overflows meets a factor of 0)
  const float da = a.m == -INFINITY ? 0.f : fmaxf(__fsub_rn(a.m, m), kLeast);
  const float db = b.m == -INFINITY ? 0.f : fmaxf(__fsub_rn(b.m, m), kLeast);
  const float fa = ex2_approx(__fmul_rn(da, kLog2e)), fb = ex2_approx(__fmul_rn(db, kLog2e));
  State c;
  c.m = m;
  c.s = __fmaf_rn(a.s, fa, __fmul_rn(b.s, fb));
  c.t = __fmaf_rn(__fmaf_rn(a.s, da, a.t), fa, __fmul_rn(__fmaf_rn(b.s, db, b.t), fb));
  return c;
}

// Logits as whole numbers in their order, equal ones alike (-0 as +0), NaN
// above all; a candidate's key also orders equal logits by the lower index.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ unsigned long long key_of(float x, int i) {
  return static_cast<unsigned long long>(order_of(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}

template <typename T>
struct Row {
  static constexpr int E = 16 / sizeof(T);  // elements of a 16-byte piece
  const T* x;
  int vocab;
  int shift;   // elements by which the row starts behind a 16-byte boundary
  int pieces;  // 16-byte pieces that the row touches; piece v holds elements v E - shift ...
  int per_seg;
  int inner0, inner1;  // pieces that lie inside the row

  __device__ Row(const void* base, long long stride, int row, int n) {
    x = static_cast<const T*>(base) + static_cast<long long>(row) * stride;
    vocab = n;
    shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    pieces = (shift + n + E - 1) / E;
    per_seg = (pieces + kSegs - 1) / kSegs;
    inner0 = shift > 0 ? 1 : 0;
    inner1 = (shift + n) / E;
  }
  __device__ static float one(const T* p) {
    if (sizeof(T) == 4) return ld_f32(reinterpret_cast<const float*>(p));
    unsigned short b;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(b) : "l"(p));
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
  }
  // Piece v as it lies in memory; elements outside the row are -inf.
  __device__ __forceinline__ uint4 load(int v) const {
    const int i0 = v * E - shift;
    if (i0 >= 0 && i0 + E <= vocab) return ld_u4(x + i0);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (sizeof(T) == 4) {
        const int at = i0 + j;
        w[j] = at >= 0 && at < vocab ? __float_as_uint(one(x + at)) : 0xff800000u;
      } else {
        const int at = i0 + 2 * j;
        const uint32_t lo = at >= 0 && at < vocab ? __float_as_uint(one(x + at)) >> 16 : 0xff80u;
        w[j] = lo | (at + 1 >= 0 && at + 1 < vocab ? __float_as_uint(one(x + at + 1)) : 0xff800000u);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ const uint4* first() const { return reinterpret_cast<const uint4*>(x - shift); }
  // The largest of the elements of pieces (bf16: two at a time).
  template <int N>
  __device__ __forceinline__ static float largest(const uint4 (&r)[N]) {
    auto more = [](uint32_t a, uint32_t b) {
      if (sizeof(T) == 4) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
      asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
      return a;
    };
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t one = more(more(r[i].x, r[i].y), more(r[i].z, r[i].w));
      m = i == 0 ? one : more(m, one);
    }
    if (sizeof(T) == 4) return __uint_as_float(m);
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ __forceinline__ static void values(const uint4& r, float (&f)[E]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (sizeof(T) == 4) {
        f[j] = __uint_as_float(w[j]);
      } else {
        f[(2 * j) % E] = __uint_as_float(w[j] << 16);
        f[(2 * j + 1) % E] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
};

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float ld_dsmem_f32(const void* p, uint32_t rank) {
  return __uint_as_float(ld_dsmem_u32(p, rank));
}

// The logit that a candidate's key was made of (-0 comes back as +0).
__device__ __forceinline__ float logit_of(unsigned long long key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(o == 0xffffffffu ? 0x7fc00000u : o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Binary tree over a power of two of states, in place; the result is a[0].
template <int N>
__device__ __forceinline__ void join_tree(State (&a)[N]) {
#pragma unroll
  for (int w = 1; w < N; w *= 2)
#pragma unroll
    for (int i = 0; i + w < N; i += 2 * w) a[i] = join(a[i], a[i + w]);
}

struct Shared {
  State state[kThreads];
  State leaf[3][kThreads];  // of a thread alone: joined states of its first half, quarter, ... of segments
  alignas(16) float best[kGroups];
  unsigned long long best_key[kGroups];
  int winners[kThreads];
  unsigned long long cand[kCap];
  unsigned long long top[kMaxTop];
  unsigned long long all[8 * kMaxTop];
  float warp_max[kWarps];
  float2 warp_sum[kWarps];
  unsigned long long bound;
  int n_winners, n_cand;
};

template <typename T, int CL>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(Args a) {
  constexpr int E = Row<T>::E, SEGS = kSegs / CL;
  griddep_launch_dependents();
  griddep_wait();
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int row = blockIdx.x / CL;
  const Row<T> x(a.logits, a.stride, row, a.vocab);

  // ---- one pass: (m, s, t) of each segment's elements of this thread, the
  // segments joined as the leaves of a binary tree; and the largest element.
  // Once a piece has been worked on its registers take the next one.
  State st = {-INFINITY, 0.f, 0.f};
  float best = -INFINITY;
  constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf throughout
  uint4 raw[P];
  // the P pieces of this thread, kThreads apart from `at` on and below `end`
  int at = rank * SEGS * x.per_seg, end = min(at + x.per_seg, x.pieces);
  auto inside = [&] { return at >= x.inner0 && min(at + kThreads * P, end) <= x.inner1; };
  const uint4* from;  // the first of them
  auto fetch = [&](int p, auto in) {
    const int w = at + tid + p * kThreads;
    raw[p] = make_uint4(kNone, kNone, kNone, kNone);
    if (w < end) raw[p] = decltype(in)::value ? ld_u4(from + p * kThreads) : x.load(w);
  };
  auto fetch_all = [&](auto in) {
    from = x.first() + at + tid;
#pragma unroll
    for (int p = 0; p < P; ++p) fetch(p, in);
  };
  if (inside()) fetch_all(Yes{});
  else fetch_all(No{});
  int id = -1;  // a given token, far ahead of its use
  if (rank == 0 && tid < a.n_tokens) id = ld_s32(a.tokens + static_cast<size_t>(row) * a.n_tokens + tid);
#pragma unroll 1
  for (int i = 0; i < SEGS;) {
    const float mt = Row<T>::largest(raw);
    if (mt > st.m) {
      if (st.m != -INFINITY) {
        const float d = fmaxf(__fsub_rn(st.m, mt), kLeast), c = ex2_approx(__fmul_rn(d, kLog2e));
        st.t = __fmul_rn(__fmaf_rn(st.s, d, st.t), c);
        st.s = __fmul_rn(st.s, c);
      }
      st.m = mt;
    }
    const float m = st.m == -INFINITY ? 0.f : st.m;
    const uint64_t log2e = pack2(kLog2e, kLog2e);
    uint64_t s2[2] = {0, 0}, t2[2] = {0, 0};
    const int here = end - at;
    at += kThreads * P;
    const bool ends = at >= end;
    if (ends) {
      at = (rank * SEGS + i + 1) * x.per_seg;
      end = i + 1 < SEGS ? min(at + x.per_seg, x.pieces) : at;
    }
    auto work = [&](auto in) {
      from = x.first() + at + tid;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float f[E];
        Row<T>::values(raw[p], f);
        fetch(p, in);
        // of no thread (those of some threads only are -inf elsewhere and add 0)
        if (p * kThreads >= here) continue;
#pragma unroll
        for (int j = 0; j < E; j += 2) {
          const uint64_t d = pack2(__fsub_rn(f[j], m), __fsub_rn(f[j + 1], m));
          const float2 y = unpack2(mul2(d, log2e)), dd = unpack2(d);
          const uint64_t e = pack2(ex2_approx(y.x), ex2_approx(y.y));
          s2[(j / 2) & 1] = add2(s2[(j / 2) & 1], e);
          // e = 0 at d = -inf: the product is 0
          t2[(j / 2) & 1] = fma2(e, pack2(fmaxf(dd.x, kLeast), fmaxf(dd.y, kLeast)), t2[(j / 2) & 1]);
        }
      }
    };
    if (inside()) work(Yes{});
    else work(No{});
    const float2 sa = unpack2(add2(s2[0], s2[1])), ta = unpack2(add2(t2[0], t2[1]));
    st.s = __fadd_rn(st.s, __fadd_rn(sa.x, sa.y));
    st.t = __fadd_rn(st.t, __fadd_rn(ta.x, ta.y));
    if (!ends) continue;
    // (where a NaN was among the elements s is one, whatever m is)
    best = fmaxf(best, st.m);
    if (SEGS > 1) {
      int level = 0;
      for (; i >> level & 1; ++level) st = join(sh.leaf[level][tid], st);
      if (level < 3) sh.leaf[level][tid] = st;
    }
    if (++i < SEGS) st = {-INFINITY, 0.f, 0.f};
  }
  const State mine = st;
  sh.state[tid] = mine;
  float given = 0.f;
  if (id >= 0 && id < a.vocab) given = Row<T>::one(x.x + id);

  // ---- the k best of this CTA's segments, in falling order in sh.top
  const int k = a.top_k;
  if (k > 0) {
    float g = best;
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((lane & 3) == 0) sh.best[tid >> 2] = g;
    if (tid < kMaxTop) sh.top[tid] = 0;
    if (tid == 0) sh.n_winners = sh.n_cand = 0;
    // fmaxf passes over a NaN: with one about, the bound goes by exact keys
    bool by_key = __syncthreads_or(mine.s != mine.s) != 0;
    // rank of each group among the groups, equal ones by the lower group
    if (tid < kGroups) {
      const float own = sh.best[tid];
      int above = 0;
#pragma unroll
      for (int i = 0; i < kGroups; i += 4) {
        const float4 o = *reinterpret_cast<const float4*>(sh.best + i);
        above += (o.x > own || (o.x == own && i < tid)) + (o.y > own || (o.y == own && i + 1 < tid)) +
                 (o.z > own || (o.z == own && i + 2 < tid)) + (o.w > own || (o.w == own && i + 3 < tid));
      }
      if (above == k - 1) sh.bound = static_cast<unsigned long long>(order_of(own)) << 32;
    }
    __syncthreads();
    bool keyed = false;
    unsigned long long top = 0;  // of this thread's keys, once they are looked at
#pragma unroll 1
    while (true) {
      if (by_key && !keyed) {
        // the exact largest key of each group's elements, and the k-th of them
        for (int v0 = rank * SEGS * x.per_seg, i = 0; i < SEGS; ++i, v0 += x.per_seg)
          for (int v = v0 + tid; v < min(v0 + x.per_seg, x.pieces); v += kThreads) {
            float f[E];
            Row<T>::values(x.load(v), f);
#pragma unroll
            for (int j = 0; j < E; ++j) {
              const int at = v * E - x.shift + j;
              if (at >= 0 && at < x.vocab) top = max(top, key_of(f[j], at));
            }
          }
        unsigned long long most = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        if ((lane & 3) == 0) sh.best_key[tid >> 2] = most;
        __syncthreads();
        if (tid < kGroups) {
          most = sh.best_key[tid];
          int above = 0;
          for (int i = 0; i < kGroups; ++i) above += sh.best_key[i] > most || (sh.best_key[i] == most && i < tid);
          if (above == k - 1) sh.bound = max(sh.bound, most);
        }
        keyed = true;
        __syncthreads();
      }
      const unsigned long long bound = sh.bound;
      if (by_key ? top >= bound && top != 0 : order_of(best) >= static_cast<uint32_t>(bound >> 32))
        sh.winners[atomicAdd(&sh.n_winners, 1)] = tid;
      __syncthreads();
      // the winners' elements at or above the bound, a piece a thread; the
      // comparison by value leaves few keys to be formed
      const float least = logit_of(bound);
      const int each = (x.per_seg + kThreads - 1) / kThreads;  // pieces of a thread in a segment
      for (int n = tid; n < sh.n_winners * SEGS * each; n += kThreads) {
        const int pair = n / each, q = n - pair * each;
        const int v0 = (rank * SEGS + pair % SEGS) * x.per_seg;
        const int v = v0 + q * kThreads + sh.winners[pair / SEGS];
        if (v >= min(v0 + x.per_seg, x.pieces)) continue;
        const uint4 piece[1] = {x.load(v)};
        if (!by_key && Row<T>::largest(piece) < least) continue;
        float f[E];
        Row<T>::values(piece[0], f);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const int at = v * E - x.shift + j;
          if (f[j] < least || at < 0 || at >= x.vocab) continue;
          const unsigned long long key = key_of(f[j], at);
          if (key >= bound) {
            const int c = atomicAdd(&sh.n_cand, 1);
            if (c < kCap) sh.cand[c] = key;
          }
        }
      }
      __syncthreads();
      const int found = sh.n_cand, n = min(found, kCap);
      // rank by counting: keys differ, so the ranks do
      for (int c = tid; c < n; c += kThreads) {
        const unsigned long long key = sh.cand[c];
        int above = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) above += sh.cand[i] > key;
        if (above < k) sh.top[above] = key;
      }
      __syncthreads();
      if (found <= kCap) break;
      // more candidates than fit: ties at the bound (many equal logits), or a
      // few groups with most of the large ones.  First find the bound by exact
      // keys, then take the k-th of those collected, which leaves at most
      // found - (kCap - k) for the next round.
      if (tid == 0) {
        if (keyed) sh.bound = sh.top[k - 1];
        sh.n_winners = sh.n_cand = 0;
      }
      by_key = true;
      __syncthreads();
    }
  }

  // ---- the row: states of the cluster's CTAs, thread by thread, then over
  // the threads; and the best of each CTA's k best
  if (CL > 1) cluster_sync();
  else __syncthreads();
  if (rank == 0) {
    State c[CL];
#pragma unroll
    for (int i = 0; i < CL; ++i) {
      if (i == 0) {
        c[i] = sh.state[tid];
      } else {
        c[i].m = ld_dsmem_f32(&sh.state[tid].m, i);
        c[i].s = ld_dsmem_f32(&sh.state[tid].s, i);
        c[i].t = ld_dsmem_f32(&sh.state[tid].t, i);
      }
    }
    unsigned long long key = 0;
    if (CL > 1 && tid < CL * k) {
      const unsigned long long* p = &sh.top[tid % k];
      const uint32_t lo = ld_dsmem_u32(p, tid / k), hi = ld_dsmem_u32(reinterpret_cast<const uint32_t*>(p) + 1, tid / k);
      key = static_cast<unsigned long long>(hi) << 32 | lo;
      sh.all[tid] = key;
    }
    join_tree(c);
    // the row's largest logit, every thread's sums for it, and their sum
    State st = c[0];
    float m = st.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sh.warp_max[warp] = m;
    __syncthreads();
    m = sh.warp_max[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) m = fmaxf(m, sh.warp_max[i]);
    const float d = st.m == -INFINITY ? 0.f : fmaxf(__fsub_rn(st.m, m), kLeast), f = ex2_approx(__fmul_rn(d, kLog2e));
    st.t = __fmul_rn(__fmaf_rn(st.s, d, st.t), f);
    st.s = __fmul_rn(st.s, f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      st.s = __fadd_rn(st.s, __shfl_xor_sync(0xffffffffu, st.s, o));
      st.t = __fadd_rn(st.t, __shfl_xor_sync(0xffffffffu, st.t, o));
    }
    if (lane == 0) sh.warp_sum[warp] = make_float2(st.s, st.t);
    __syncthreads();
    float sum = sh.warp_sum[0].x, sum_t = sh.warp_sum[0].y;
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
      sum = __fadd_rn(sum, sh.warp_sum[i].x);
      sum_t = __fadd_rn(sum_t, sh.warp_sum[i].y);
    }
    const float log_s = logf(sum);
    if (a.entropy && tid == 0) a.entropy[row] = __fsub_rn(log_s, __fdiv_rn(sum_t, sum));
    auto log_prob = [&](float logit) { return __fsub_rn(__fsub_rn(logit, m), log_s); };
    if (id >= a.vocab) flag_error(a.status, kStatusIndex);
    if (id >= 0 && id < a.vocab) a.token_lp[static_cast<size_t>(row) * a.n_tokens + tid] = log_prob(given);
    for (int j = tid + kThreads; j < a.n_tokens; j += kThreads) {
      const size_t at = static_cast<size_t>(row) * a.n_tokens + j;
      const int more = ld_s32(a.tokens + at);
      if (more >= a.vocab) flag_error(a.status, kStatusIndex);
      if (more >= 0 && more < a.vocab) a.token_lp[at] = log_prob(Row<T>::one(x.x + more));
    }
    auto put = [&](int at, unsigned long long best_key) {
      const size_t to = static_cast<size_t>(row) * k + at;
      a.top_ids[to] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best_key));
      a.top_lp[to] = log_prob(logit_of(best_key));
    };
    if (CL == 1) {
      if (tid < k) put(tid, sh.top[tid]);
    } else if (tid < CL * k && key != 0) {
      int above = 0;
      for (int i = 0; i < CL * k; ++i) above += sh.all[i] > key;
      if (above < k) put(above, key);
    }
  }
  if (CL > 1) cluster_sync();  // this CTA's shared memory has been read
}

template <typename T, int CL>
hb_status logprobs_launch(const Args& a, int rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * CL);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  const hb_status st = cuda_status(cudaLaunchKernelEx(&cfg, logprobs_kernel<T, CL>, a), "logprobs_kernel launch");
  if (st == HB_OK) count_launch();
  return st;
}

template <typename T>
hb_status logprobs_rows(const Args& a, int rows, int num_sms, cudaStream_t stream) {
  // As many CTAs a row as keep the grid within four a SM, which is what is resident
  // at a time.  Measured, fp32 rows of 32000 (L2 flushed, with the launch): 160 rows
  // 19 us with 2 CTAs a row, 25 with 4, 33 with 8; 512 rows 28 with 1, 35 with 2.
  const long long room = 4ll * num_sms;
  if (rows * 8ll <= room) return logprobs_launch<T, 8>(a, rows, stream);
  if (rows * 4ll <= room) return logprobs_launch<T, 4>(a, rows, stream);
  if (rows * 2ll <= room) return logprobs_launch<T, 2>(a, rows, stream);
  return logprobs_launch<T, 1>(a, rows, stream);
}

}  // namespace
}  // namespace hb

extern "C" hb_status hb_logprobs(const void* logits, int32_t logits_type, int32_t n_rows, int32_t vocab,
                                 int64_t row_stride, const int32_t* tokens, int32_t n_tokens, float* token_logprobs,
                                 float* entropy, int32_t top_k, int32_t* top_ids, float* top_logprobs, void* stream) {
  using namespace hb;
  clear_error();
  HB_REQUIRE(logits_type == HB_LOGITS_F32 || logits_type == HB_LOGITS_BF16, "hb_logprobs: unknown logits type %d",
             logits_type);
  HB_REQUIRE(n_rows >= 0 && vocab > 0 && row_stride >= vocab, "hb_logprobs: n_rows >= 0, vocab > 0, row_stride >= vocab");
  HB_REQUIRE(vocab <= (1 << 30) && n_rows <= (1 << 28), "hb_logprobs: at most 2^30 logits a row and 2^28 rows");
  HB_REQUIRE(n_tokens >= 0, "hb_logprobs: n_tokens >= 0");
  HB_REQUIRE(top_k >= 0 && top_k <= vocab && top_k <= kMaxTop, "hb_logprobs: top_k must be in 0 .. min(vocab, %d)",
             kMaxTop);
  if (n_rows == 0) return HB_OK;
  HB_REQUIRE(logits != nullptr, "hb_logprobs: null pointer");
  HB_REQUIRE(n_tokens == 0 || (tokens && token_logprobs), "hb_logprobs: null tokens or token_logprobs");
  HB_REQUIRE(top_k == 0 || (top_ids && top_logprobs), "hb_logprobs: null top_ids or top_logprobs");
  HB_REQUIRE((reinterpret_cast<uintptr_t>(logits) & (logits_type == HB_LOGITS_F32 ? 3u : 1u)) == 0 && aligned4(tokens) &&
                 aligned4(token_logprobs) && aligned4(entropy) && aligned4(top_ids) && aligned4(top_logprobs),
             "hb_logprobs: operands aligned to their elements");
  if (n_tokens == 0 && top_k == 0 && !entropy) return HB_OK;
  DeviceCtx ctx;
  hb_status st = device_context(&ctx);
  if (st != HB_OK) return st;
  const Args a = {logits, row_stride, vocab, tokens, n_tokens, token_logprobs, entropy, top_k, top_ids, top_logprobs,
                  ctx.status};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return logits_type == HB_LOGITS_F32 ? logprobs_rows<float>(a, n_rows, ctx.num_sms, s)
                                      : logprobs_rows<__nv_bfloat16>(a, n_rows, ctx.num_sms, s);
}
