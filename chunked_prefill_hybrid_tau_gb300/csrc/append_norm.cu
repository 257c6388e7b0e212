// Per-head RMS norm of queries and keys, RoPE and the paged K/V append in
// one pass over the packed rows (the layer of models with normed q/k heads;
// without the norm: kv_append_kernel in elementwise.cu).
//
// For head vector x (d = d_head elements) of a q or k head at position p:
//   y = x / sqrt(mean(x^2) + eps) * g              (g_q or g_k, fp32)
//   out_i = y_i cos_i - y_{i+d/2} sin_i,  out_{i+d/2} = y_{i+d/2} cos_i + y_i sin_i
// rounded once to bf16: neither the normed nor the rotated head is stored in
// between.  q goes to its row, K and the raw V to the row's slot.
//
// Reads T (n_q + 2 n_kv) d bf16 and writes as much: HBM bounds it (one read
// and one write of the projection's output).
#include <cuda_bf16.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace {

using namespace dev;

// A CTA takes one row at a time, rows gridDim.x apart.  A thread owns 8
// elements of a head's first half and the matching 8 of its second half, so
// the rotation stays in the thread and the norm's sum is a shuffle among the
// head's d / 16 neighbouring lanes; V heads take the same pieces and copy
// them.  Each thread has U = 2 heads (half the heads apart) in flight and one
// set of (cos, sin) for both; the row's q, k and v pieces do not wait for its
// position and slot, and those of the next row are fetched ahead.  Measured,
// 8192 rows of 72 heads of 128 (floor 45.3 us at the copy rate): 82.7 us with
// a CTA per row and one head a thread, 52.3 us this way at 72 registers (56
// registers spill: 76 us; 3 heads a thread: 64 us).
constexpr int U = 2;
constexpr int kMaxThreads = 512;
constexpr int kRegs = 72;

template <int DH>
__global__ void __maxnreg__(kRegs)
    kv_append_norm_kernel(const __nv_bfloat16* qkv, const int* row_pos, const int* slots, const float2* rope, int T,
                          int max_pos, int n_q, int n_kv, const __nv_bfloat16* g_q, const __nv_bfloat16* g_k, float eps,
                          __nv_bfloat16* q_out, __nv_bfloat16* kc, __nv_bfloat16* vc, long long num_slots, int* status,
                          int* zero, int n_zero) {
  constexpr int HALF = DH / 2;
  constexpr int RC = HALF / 8;  // threads per head
  griddep_launch_dependents();
  griddep_wait();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n_zero; i += gridDim.x * blockDim.x) zero[i] = 0;
  const int heads = n_q + 2 * n_kv;
  const int c = threadIdx.x % RC;
  const int hp = blockDim.x / RC;  // heads of one pass of the CTA
  // the lanes of one head; they take every branch below together
  const unsigned group = ((1u << RC) - 1u) << ((threadIdx.x & 31) & ~(RC - 1));
  int r = blockIdx.x;
  int pos = ld_s32(row_pos + r), slot = ld_s32(slots + r);
  while (r < T) {
    const __nv_bfloat16* src_row = qkv + static_cast<size_t>(r) * heads * DH + c * 8;
    const bool pos_ok = pos >= 0 && pos < max_pos;
    const bool slot_ok = slot >= 0 && slot < num_slots;
    if (threadIdx.x == 0 && (!pos_ok || slot >= num_slots)) flag_error(status, kStatusIndex);
    const int page = slot / 16, off = slot % 16;
    const int r_next = r + gridDim.x;
    int pos_next = 0, slot_next = 0;
    float4 cs[4];
    for (int h0 = threadIdx.x / RC; h0 < heads; h0 += U * hp) {
      uint4 a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * hp;
        if (h < heads) {
          a[u] = ld_u4(src_row + h * DH);
          b[u] = ld_u4(src_row + h * DH + HALF);
        }
      }
      if (!pos_ok) break;
      if (h0 < hp) {
        const float2* csp = rope + static_cast<size_t>(pos) * HALF + c * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) cs[j] = ld_f4(csp + 2 * j);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * hp;
        if (h >= heads || (h >= n_q && !slot_ok)) continue;
        __nv_bfloat16* dst;
        if (h < n_q)
          dst = q_out + (static_cast<size_t>(r) * n_q + h) * DH;
        else if (h < n_q + n_kv)
          dst = kc + ((static_cast<size_t>(page) * n_kv + (h - n_q)) * 16 + off) * DH;
        else
          dst = vc + ((static_cast<size_t>(page) * n_kv + (h - n_q - n_kv)) * 16 + off) * DH;
        uint4 o1 = a[u], o2 = b[u];
        if (h < n_q + n_kv) {
          const __nv_bfloat16* g = (h < n_q ? g_q : g_k) + c * 8;
          const uint4 ga = ld_u4(g), gb = ld_u4(g + HALF);
          const uint32_t aw[4] = {o1.x, o1.y, o1.z, o1.w}, bw[4] = {o2.x, o2.y, o2.z, o2.w};
          const uint32_t gaw[4] = {ga.x, ga.y, ga.z, ga.w}, gbw[4] = {gb.x, gb.y, gb.z, gb.w};
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x1 = unpack_bf16x2(aw[j]), x2 = unpack_bf16x2(bw[j]);
            ss = __fmaf_rn(x1.x, x1.x, ss);
            ss = __fmaf_rn(x1.y, x1.y, ss);
            ss = __fmaf_rn(x2.x, x2.x, ss);
            ss = __fmaf_rn(x2.y, x2.y, ss);
          }
#pragma unroll
          for (int o = RC / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
          const float inv = rsqrtf(ss * (1.0f / DH) + eps);
          uint32_t w1[4], w2[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 t = cs[j];  // (cos, sin) of elements 2j and 2j + 1
            const float2 x1 = unpack_bf16x2(aw[j]), x2 = unpack_bf16x2(bw[j]);
            const float2 g1 = unpack_bf16x2(gaw[j]), g2 = unpack_bf16x2(gbw[j]);
            const float p0 = x1.x * inv * g1.x, p1 = x1.y * inv * g1.y;
            const float s0 = x2.x * inv * g2.x, s1 = x2.y * inv * g2.y;
            w1[j] = pack_bf16x2(p0 * t.x - s0 * t.y, p1 * t.z - s1 * t.w);
            w2[j] = pack_bf16x2(s0 * t.x + p0 * t.y, s1 * t.z + p1 * t.w);
          }
          o1 = make_uint4(w1[0], w1[1], w1[2], w1[3]);
          o2 = make_uint4(w2[0], w2[1], w2[2], w2[3]);
        }
        *reinterpret_cast<uint4*>(dst + c * 8) = o1;
        *reinterpret_cast<uint4*>(dst + HALF + c * 8) = o2;
      }
    }
    if (r_next < T) {
      pos_next = ld_s32(row_pos + r_next);
      slot_next = ld_s32(slots + r_next);
    }
    r = r_next;
    pos = pos_next;
    slot = slot_next;
  }
}

}  // namespace

hb_status kv_append_norm_launch(const DeviceCtx& ctx, const void* qkv, int T, const int* row_pos, const int* slots,
                                const void* rope, int max_pos, const hb_layer_dims& dm, const void* g_q,
                                const void* g_k, void* q_out, void* k_cache, void* v_cache, int num_pages,
                                cudaStream_t stream, int* zero, int n_zero) {
  // a CTA's threads cover the row's heads in one pass of U heads each
  const int heads = dm.n_q + 2 * dm.n_kv, rc = dm.d_head / 16;
  int threads = (heads + U - 1) / U * rc;
  threads = threads < kMaxThreads ? (threads + 31) / 32 * 32 : kMaxThreads;
  // as many CTAs as are resident at a time, no more: a partial second wave
  // left a third of the SMs idle (74 against 60 us for 8192 rows)
  const int fit = 65536 / (kRegs * threads);
  const int per_sm = fit < 16 ? fit : 16;
  const int grid = T < ctx.num_sms * per_sm ? T : ctx.num_sms * per_sm;
  const long long num_slots = static_cast<long long>(num_pages) * 16;
  auto* in = static_cast<const __nv_bfloat16*>(qkv);
  auto* gq = static_cast<const __nv_bfloat16*>(g_q);
  auto* gk = static_cast<const __nv_bfloat16*>(g_k);
  auto* qo = static_cast<__nv_bfloat16*>(q_out);
  auto* kc = static_cast<__nv_bfloat16*>(k_cache);
  auto* vc = static_cast<__nv_bfloat16*>(v_cache);
  auto* rp = static_cast<const float2*>(rope);
  auto kernel = dm.d_head == 128 ? kv_append_norm_kernel<128> : kv_append_norm_kernel<64>;
  return launch_pdl(kernel, grid, threads, 0, stream, "kv_append_norm_kernel launch", in, row_pos, slots, rp, T, max_pos,
                    dm.n_q, dm.n_kv, gq, gk, dm.rms_eps, qo, kc, vc, num_slots, ctx.status, zero, n_zero);
}

}  // namespace hb

extern "C" hb_status hb_kv_append_norm(const void* qkv, int32_t T, const int32_t* row_pos, const int32_t* slot_mapping,
                                       const void* rope, int32_t max_pos, const hb_layer_dims* dims, const void* g_q,
                                       const void* g_k, void* q_out, void* k_cache, void* v_cache, int32_t num_pages,
                                       void* stream) {
  hb::clear_error();
  hb_status st = hb::check_dims(dims);
  if (st != HB_OK) return st;
  HB_REQUIRE(T >= 0 && max_pos > 0 && num_pages > 0, "hb_kv_append_norm: bad sizes");
  if (T == 0) return HB_OK;
  HB_REQUIRE(qkv && row_pos && slot_mapping && rope && g_q && g_k && q_out && k_cache && v_cache,
             "hb_kv_append_norm: null pointer");
  HB_REQUIRE(hb::aligned16(qkv) && hb::aligned16(q_out) && hb::aligned16(k_cache) && hb::aligned16(v_cache) &&
                 hb::aligned16(rope) && hb::aligned16(g_q) && hb::aligned16(g_k),
             "hb_kv_append_norm: 16-byte alignment");
  hb::DeviceCtx ctx;
  st = hb::device_context(&ctx);
  if (st != HB_OK) return st;
  return hb::kv_append_norm_launch(ctx, qkv, T, row_pos, slot_mapping, rope, max_pos, *dims, g_q, g_k, q_out, k_cache,
                                   v_cache, num_pages, static_cast<cudaStream_t>(stream));
}
