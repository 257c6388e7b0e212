// RoPE and the paged K/V append into a cache of E4M3 codes (with or without
// the per-head RMS norm of queries and keys), one pass over the packed rows.
//
// Per head vector of a q or k head at position p, as in append_norm.cu:
//   y = x, or x / sqrt(mean(x^2) + eps) * g
//   out_i = y_i cos_i - y_{i+d/2} sin_i,  out_{i+d/2} = y_{i+d/2} cos_i + y_i sin_i
// q is rounded to bf16.  A key's out and a raw value vector z are quantized:
//   amax = max |z|,  e = least integer >= -100 with amax <= 448 * 2^e,
//   code = E4M3(z * 2^-e), scale byte e + 127.
// A power of two is as good a scale as amax / 448 (a floating-point code's
// relative step does not depend on the scale, and codes that fall below the
// smallest normal one are 2^-14 of the largest), and it makes code * 2^e exact
// in bf16, so the attention reads the cache without a second rounding.  The
// floor -100 keeps the smallest code's value, 2^-109, a normal number.
//
// Reads T (n_q + 2 n_kv) d bf16 and writes T n_q d bf16 and 2 T n_kv (d + 1)
// bytes: HBM bounds it.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace {

using namespace dev;

// The work split is kv_append_norm_kernel's: a CTA takes one row at a time; a
// thread owns 8 elements of a head's first half and the matching 8 of its
// second half, so the rotation stays in the thread, and the norm's sum and the
// maximum are shuffles among the head's d / 16 neighbouring lanes; two heads
// in flight a thread.  8192 rows of 72 heads of 128 (floor 43.3 us at the copy
// rate): 46.5 us at 72 registers, as many CTAs as fit; 50.5 at 64, 56.7 at 56,
// 53.8 at 80.
// Normed they take 54.2 (the gains are loaded for every head, 4 bytes spill); rows of
// 64 + 16 heads, which make 20 warps an SM, 57.9 and normed 67.9 (floor 48.3).
constexpr int U = 2;
constexpr int kMaxThreads = 512;
constexpr int kRegs = 72;
constexpr int kMinExp = -100;

__device__ __forceinline__ uint2 codes8(const float (&y)[8], float f) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j] * f, y[2 * j + 1] * f), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <int DH, bool NORM>
__global__ void __maxnreg__(kRegs)
    kv_append_e4m3_kernel(const __nv_bfloat16* qkv, const int* row_pos, const int* slots, const float2* rope, int T,
                          int max_pos, int n_q, int n_kv, const __nv_bfloat16* g_q, const __nv_bfloat16* g_k, float eps,
                          __nv_bfloat16* q_out, uint8_t* kc, uint8_t* ks, uint8_t* vc, uint8_t* vs, long long num_slots,
                          int* status) {
  constexpr int HALF = DH / 2;
  constexpr int RC = HALF / 8;  // threads per head
  griddep_launch_dependents();
  griddep_wait();
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
        const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
        float y1[8], y2[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x1 = unpack_bf16x2(aw[j]), x2 = unpack_bf16x2(bw[j]);
          y1[2 * j] = x1.x, y1[2 * j + 1] = x1.y;
          y2[2 * j] = x2.x, y2[2 * j + 1] = x2.y;
        }
        if (h < n_q + n_kv) {
          if (NORM) {
            const __nv_bfloat16* g = (h < n_q ? g_q : g_k) + c * 8;
            const uint4 ga = ld_u4(g), gb = ld_u4(g + HALF);
            const uint32_t gaw[4] = {ga.x, ga.y, ga.z, ga.w}, gbw[4] = {gb.x, gb.y, gb.z, gb.w};
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __fmaf_rn(y1[j], y1[j], ss);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __fmaf_rn(y2[j], y2[j], ss);
#pragma unroll
            for (int o = RC / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
            const float inv = rsqrtf(ss * (1.0f / DH) + eps);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 g1 = unpack_bf16x2(gaw[j]), g2 = unpack_bf16x2(gbw[j]);
              y1[2 * j] = y1[2 * j] * inv * g1.x, y1[2 * j + 1] = y1[2 * j + 1] * inv * g1.y;
              y2[2 * j] = y2[2 * j] * inv * g2.x, y2[2 * j + 1] = y2[2 * j + 1] * inv * g2.y;
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float cosj = (j & 1) ? cs[j / 2].z : cs[j / 2].x, sinj = (j & 1) ? cs[j / 2].w : cs[j / 2].y;
            const float p = y1[j], s = y2[j];
            y1[j] = p * cosj - s * sinj;
            y2[j] = s * cosj + p * sinj;
          }
        }
        if (h < n_q) {
          __nv_bfloat16* dst = q_out + (static_cast<size_t>(r) * n_q + h) * DH + c * 8;
          *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(y1[0], y1[1]), pack_bf16x2(y1[2], y1[3]),
                                                      pack_bf16x2(y1[4], y1[5]), pack_bf16x2(y1[6], y1[7]));
          *reinterpret_cast<uint4*>(dst + HALF) = make_uint4(pack_bf16x2(y2[0], y2[1]), pack_bf16x2(y2[2], y2[3]),
                                                             pack_bf16x2(y2[4], y2[5]), pack_bf16x2(y2[6], y2[7]));
          continue;
        }
        // the magnitudes' bit patterns order as their values do, NaN above all
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m = max(m, __float_as_uint(y1[j]) & 0x7fffffffu);
          m = max(m, __float_as_uint(y2[j]) & 0x7fffffffu);
        }
#pragma unroll
        for (int o = RC / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(group, m, o));
        // 448 = 1.75 * 2^8: the exponent of amax less 8, one more where its
        // mantissa is above 1.75
        const int e = max(static_cast<int>((m + 0x1fffffu) >> 23) - 135, kMinExp);
        const bool finite = m < 0x7f800000u;
        const float f = __uint_as_float(finite ? static_cast<uint32_t>(127 - e) << 23 : 0x7fc00000u);
        const bool is_v = h >= n_q + n_kv;
        const size_t at = (static_cast<size_t>(page) * n_kv + (h - n_q - (is_v ? n_kv : 0))) * 16 + off;
        uint8_t* dst = (is_v ? vc : kc) + at * DH + c * 8;
        *reinterpret_cast<uint2*>(dst) = codes8(y1, f);
        *reinterpret_cast<uint2*>(dst + HALF) = codes8(y2, f);
        if (c == 0) (is_v ? vs : ks)[at] = static_cast<uint8_t>(finite ? e + 127 : 255);
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
}  // namespace hb

extern "C" hb_status hb_kv_append_e4m3(const void* qkv, int32_t T, const int32_t* row_pos, const int32_t* slot_mapping,
                                       const void* rope, int32_t max_pos, const hb_layer_dims* dims, const void* g_q,
                                       const void* g_k, void* q_out, void* k_cache, void* k_scale, void* v_cache,
                                       void* v_scale, int32_t num_pages, void* stream) {
  using namespace hb;
  clear_error();
  hb_status st = check_dims(dims);
  if (st != HB_OK) return st;
  HB_REQUIRE(T >= 0 && max_pos > 0 && num_pages > 0, "hb_kv_append_e4m3: bad sizes");
  if (T == 0) return HB_OK;
  HB_REQUIRE(qkv && row_pos && slot_mapping && rope && q_out && k_cache && k_scale && v_cache && v_scale,
             "hb_kv_append_e4m3: null pointer");
  HB_REQUIRE((g_q == nullptr) == (g_k == nullptr), "hb_kv_append_e4m3: one of the gains g_q, g_k without the other");
  HB_REQUIRE(aligned16(qkv) && aligned16(q_out) && aligned16(k_cache) && aligned16(v_cache) && aligned16(rope) &&
                 aligned16(g_q) && aligned16(g_k),
             "hb_kv_append_e4m3: 16-byte alignment");
  DeviceCtx ctx;
  st = device_context(&ctx);
  if (st != HB_OK) return st;
  const hb_layer_dims& dm = *dims;
  // a CTA's threads cover the row's heads in one pass of U heads each
  const int heads = dm.n_q + 2 * dm.n_kv, rc = dm.d_head / 16;
  int threads = (heads + U - 1) / U * rc;
  threads = threads < kMaxThreads ? (threads + 31) / 32 * 32 : kMaxThreads;
  // as many CTAs as are resident at a time
  const int fit = 65536 / (kRegs * threads);
  const int per_sm = fit < 16 ? fit : 16;
  const int grid = T < ctx.num_sms * per_sm ? T : ctx.num_sms * per_sm;
  const long long num_slots = static_cast<long long>(num_pages) * 16;
  auto kernel = dm.d_head == 128 ? (g_q ? kv_append_e4m3_kernel<128, true> : kv_append_e4m3_kernel<128, false>)
                                 : (g_q ? kv_append_e4m3_kernel<64, true> : kv_append_e4m3_kernel<64, false>);
  return launch_pdl(kernel, grid, threads, 0, static_cast<cudaStream_t>(stream), "kv_append_e4m3_kernel launch",
                    static_cast<const __nv_bfloat16*>(qkv), row_pos, slot_mapping, static_cast<const float2*>(rope), T,
                    max_pos, dm.n_q, dm.n_kv, static_cast<const __nv_bfloat16*>(g_q),
                    static_cast<const __nv_bfloat16*>(g_k), dm.rms_eps, static_cast<__nv_bfloat16*>(q_out),
                    static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(k_scale), static_cast<uint8_t*>(v_cache),
                    static_cast<uint8_t*>(v_scale), num_slots, ctx.status);
}
