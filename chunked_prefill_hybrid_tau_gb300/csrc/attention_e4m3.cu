// Paged attention over a cache of E4M3 codes with a power-of-two scale per
// token and kv head (append_e4m3.cu).
//
//   out = sum_j P_j 2^ev_j V_j / sum_j P_j,  P_j = exp(2^ek_j (q . K_j) / sqrt(d) - m)
//
// One warp takes one row and q head, lanes share the head dimension, keys one
// after another with a running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace {

using namespace dev;

constexpr int kMaxSeqs = 1024;

struct Params {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const uint8_t *k, *ks, *v, *vs;
  const int* q_start;
  const int* kv_len;
  const int* block_table;
  int S, T, max_pages, num_pages, n_q, n_kv, grp, max_kv_len;
  float scale_log2;
  int* status;
};

__device__ __forceinline__ float code_value(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

__device__ __forceinline__ float scale_value(uint8_t b) {
  return __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : static_cast<uint32_t>(b) << 23);
}

template <int D>
__global__ void __launch_bounds__(128) attention_e4m3_kernel(Params p) {
  constexpr int E = D / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, row = blockIdx.x;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (row == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < p.S; i += blockDim.x)
      if (ld_s32(p.q_start + i + 1) <= ld_s32(p.q_start + i)) flag_error(p.status, kStatusIndex);
  if (h >= p.n_q) return;
  int lo = 0, hi = p.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ld_s32(p.q_start + mid) <= row) lo = mid; else hi = mid - 1;
  }
  const int s = lo, q1 = ld_s32(p.q_start + s + 1), kvl = ld_s32(p.kv_len + s);
  const int last = kvl - (q1 - row);
  if (row < ld_s32(p.q_start + s) || row >= q1 || last < 0 || kvl > p.max_kv_len || (kvl + 15) / 16 > p.max_pages) {
    flag_error(p.status, kStatusIndex);
    return;
  }
  const int g = h / p.grp;
  const int* bt = p.block_table + static_cast<size_t>(s) * p.max_pages;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(p.q[(static_cast<size_t>(row) * p.n_q + h) * D + lane * E + i]);
    o[i] = 0.f;
  }
  for (int j = 0; j <= last; ++j) {
    int page = ld_s32(bt + j / 16);
    if (page < 0 || page >= p.num_pages) {
      flag_error(p.status, kStatusIndex);
      page = 0;
    }
    const size_t at = (static_cast<size_t>(page) * p.n_kv + g) * 16 + j % 16;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) x += q[i] * code_value(p.k[at * D + lane * E + i]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= scale_value(p.ks[at]) * p.scale_log2;
    const float mn = fmaxf(m, x);
    const float alpha = exp2f(m - mn), e = exp2f(x - mn);
    m = mn;
    l = l * alpha + e;
    const float w = e * scale_value(p.vs[at]);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * alpha + w * code_value(p.v[at * D + lane * E + i]);
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    p.out[(static_cast<size_t>(row) * p.n_q + h) * D + lane * E + i] = __float2bfloat16(o[i] / l);
}

size_t workspace_bytes(const hb_layer_dims& dm, int max_seqs, int max_kv_len) {
  (void)dm, (void)max_seqs, (void)max_kv_len;
  return 256;
}

}  // namespace
}  // namespace hb

extern "C" size_t hb_attention_e4m3_workspace_bytes(const hb_layer_dims* dims, int32_t max_rows, int32_t max_seqs,
                                                    int32_t max_kv_len) {
  (void)max_rows;
  if (!dims || max_seqs < 0 || max_kv_len < 0) return 0;
  return hb::workspace_bytes(*dims, max_seqs, max_kv_len);
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
  HB_REQUIRE(max_kv_len >= 1 && num_pages > 0, "hb_attention_e4m3: max_kv_len and num_pages must be positive");
  if (plan->n_seqs == 0 || plan->n_rows == 0) return HB_OK;
  HB_REQUIRE(q && k_cache && k_scale && v_cache && v_scale && out, "hb_attention_e4m3: null pointer");
  HB_REQUIRE(plan->seq_q_start && plan->seq_kv_len && plan->block_table, "hb_attention_e4m3: null plan array");
  HB_REQUIRE(plan->n_rows >= plan->n_seqs, "hb_attention_e4m3: every sequence has at least one row (%d rows, %d sequences)",
             plan->n_rows, plan->n_seqs);
  HB_REQUIRE(aligned16(q) && aligned16(out) && aligned16(k_cache) && aligned16(v_cache) && aligned16(k_scale) &&
                 aligned16(v_scale),
             "hb_attention_e4m3: 16-byte alignment");
  const size_t need = workspace_bytes(*dims, plan->n_seqs, max_kv_len);
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
  return launch_pdl(dims->d_head == 128 ? attention_e4m3_kernel<128> : attention_e4m3_kernel<64>,
                    dim3(plan->n_rows, (dims->n_q + 3) / 4), 128, 0, static_cast<cudaStream_t>(stream),
                    "attention_e4m3_kernel launch", p);
}
