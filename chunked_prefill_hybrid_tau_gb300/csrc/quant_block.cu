// Block-scaled E4M3 quantization of bf16 matrices: the operand preparation
// of the projections with one scale per 128 columns of a token row and per
// 128 x 128 block of a weight (gemm_e4m3_block.cu).
//
// Per group (1 x 128 or 128 x 128 elements, smaller at the edges):
//   amax = max |x|,  top = max(amax, 2^-112),
//   inv = 448 / top,  scale = top / 448  (correctly rounded fp32 divisions),
//   code = E4M3(fp32(x * inv)), nearest even, saturating;
// a group of zeros gets scale 0 and zero codes.  The floor 2^-112 keeps inv
// (2^120.8) and scale (2^-120.8) normal fp32 numbers: without it 448 / amax
// is infinite for amax below 2^-119.2 and a zero beside such a value becomes
// 0 * inf = NaN.  The formulas hold for a NaN and an infinity too: a NaN
// makes its group's scale and codes NaN, an infinity makes the scale
// infinite, its own code NaN and the others zero; other groups do not notice.
//
// Both kernels read 2 bytes and write 1 byte an element once, so HBM bounds
// them if the instructions an element stay few.  With fp32 maxima and two
// divisions for every group and lane the token kernel took 66.4 us for 8192 x
// 14336 (52.6 at the copy rate), most of it issuing.  So the maximum runs
// over the bit patterns, two at a time (the magnitudes of bf16 numbers order
// as their bits do, NaN above all), and a lane divides for one group only.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr float kAmaxMin = 0x1p-112f;
constexpr int kMaxRows = 65535 * 128;  // grid limit of the block kernel
constexpr int kMaxCols = 1 << 24;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi, float inv) {
  const __nv_fp8x2_storage_t v =
      __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(lo, inv), __fmul_rn(hi, inv)), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(v);
}

// Maxima of the magnitudes of two bf16 numbers, as bit patterns.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  return max2(max2(v.x & kMag, v.y & kMag), max2(v.z & kMag, v.w & kMag));
}
// The larger of the two, as fp32.
__device__ __forceinline__ float amax_value(uint32_t m) {
  const uint32_t hi = m & 0xffff0000u, lo = m << 16;
  return __uint_as_float(hi > lo ? hi : lo);
}

__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_bf16x2(w[j]);
    b[j] = e4m3x2(f.x, f.y, inv);
  }
  return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
}

struct GroupScale {
  float inv, scale;
};
__device__ __forceinline__ GroupScale group_scale(float amax) {
  if (amax == 0.f) return {0.f, 0.f};
  const float top = amax < kAmaxMin ? kAmaxMin : amax;  // a NaN stays
  return {__fdiv_rn(448.0f, top), __fdiv_rn(top, 448.0f)};
}

// Tokens: 16 lanes own one group (16 bytes of bf16 each), so the group's
// maximum is four shuffles and no group meets another.  A CTA's 16 half
// warps cover 2^gshift groups of 16 >> gshift rows; each takes U groups,
// 2^gshift apart, with all loads in flight.
// (40 registers, six CTAs an SM: 55.0 us for 8192 x 14336; 42, five: 57.3.)
template <int U>
__global__ void __maxnreg__(40)
    quant_groups_kernel(const uint4* x, uint2* q, float* scale, int rows, int c8, int kb, int gshift) {
  griddep_launch_dependents();
  griddep_wait();
  const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int row = blockIdx.x * (16 >> gshift) + (sub >> gshift);
  const int g0 = (blockIdx.y * U << gshift) + (sub & ((1 << gshift) - 1));
  const bool row_ok = row < rows;
  const size_t base = static_cast<size_t>(row) * c8;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (g0 + (u << gshift)) * 16 + l;
    v[u] = row_ok && i < c8 ? ld_u4(x + base + i) : make_uint4(0, 0, 0, 0);
  }
  uint32_t m[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    m[u] = amax8(v[u]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m[u] = max2(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
  }
  // lane l of the group divides for group l % U and hands the factor round
  uint32_t mine = m[0];
#pragma unroll
  for (int u = 1; u < U; ++u) mine = l % U == u ? m[u] : mine;
  const GroupScale gs = group_scale(amax_value(mine));
  const int g_mine = g0 + (l << gshift);
  if (row_ok && l < U && g_mine < kb) scale[static_cast<size_t>(row) * kb + g_mine] = gs.scale;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float inv = __shfl_sync(0xffffffffu, gs.inv, u, 16);
    const int i = (g0 + (u << gshift)) * 16 + l;
    if (row_ok && i < c8) q[base + i] = codes8(v[u], inv);
  }
}

// Weights: one CTA per 128 x 128 block, held in registers (8 pieces of 16
// bytes a thread) between its maximum and its codes.
// (64 registers, four CTAs an SM: 51.8 us for 28672 x 4096, the copy rate;
// 89 registers, two: 61.2.)
__global__ void __maxnreg__(64)
    quant_blocks_kernel(const uint4* x, uint2* q, float* scale, int rows, int c8, int kb) {
  griddep_wait();
  __shared__ uint32_t red[kThreads / 32];
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int i = blockIdx.x * 16 + l;
  const int row0 = blockIdx.y * 128 + r0;
  uint4 v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int r = row0 + 16 * u;
    v[u] = r < rows && i < c8 ? ld_u4(x + static_cast<size_t>(r) * c8 + i) : make_uint4(0, 0, 0, 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) m = max2(m, amax8(v[u]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = max2(m, red[w]);
  const GroupScale gs = group_scale(amax_value(m));
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int r = row0 + 16 * u;
    if (r < rows && i < c8) q[static_cast<size_t>(r) * c8 + i] = codes8(v[u], gs.inv);
  }
  if (threadIdx.x == 0) scale[static_cast<size_t>(blockIdx.y) * kb + blockIdx.x] = gs.scale;
}

// Rows that an RMSNorm goes over before their projection (the layer's x and
// h): the token kernel's codes, and scales that carry the row's 1/rms,
//   scale[r][b] = fl(scale_b * rsqrt(mean(x[r]^2) + eps)),
// so that the projection needs no statistics (the gain is in its weights).
// One CTA per row, which it holds in registers: thread t has the 16-byte
// pieces t, t + 256, ...; groups lie in 16 neighbouring lanes as above.  The
// sum of squares is formed in an order of the row length alone.  Also clears
// n_zero ints (the layer's counters).
template <int NV>
__global__ void __launch_bounds__(kThreads)
    quant_norm_kernel(const uint4* x, uint2* q, float* scale, int c8, int kb, float inv_d, float eps, int* zero,
                      int n_zero) {
  griddep_launch_dependents();
  griddep_wait();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n_zero; i += gridDim.x * blockDim.x) zero[i] = 0;
  __shared__ float red[kThreads / 32];
  const int t = threadIdx.x, l = t & 15;
  const size_t base = static_cast<size_t>(blockIdx.x) * c8;
  uint4 v[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = t + kThreads * k;
    v[k] = i < c8 ? ld_u4(x + base + i) : make_uint4(0, 0, 0, 0);
  }
  float ss = 0.f;
  uint32_t m[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_bf16x2(w[j]);
      ss = __fmaf_rn(f.x, f.x, ss);
      ss = __fmaf_rn(f.y, f.y, ss);
    }
    m[k] = amax8(v[k]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m[k] = max2(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
  if ((t & 31) == 0) red[t >> 5] = ss;
  __syncthreads();
  ss = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) ss = __fadd_rn(ss, red[w]);
  const float inv_rms = rsqrtf(__fmaf_rn(ss, inv_d, eps));
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = t + kThreads * k;
    if (i >= c8) break;
    const GroupScale gs = group_scale(amax_value(m[k]));
    q[base + i] = codes8(v[k], gs.inv);
    if (l == 0) scale[static_cast<size_t>(blockIdx.x) * kb + i / 16] = __fmul_rn(gs.scale, inv_rms);
  }
}

}  // namespace

hb_status quant_norm_launch(const DeviceCtx& ctx, const void* x, void* q, float* scale, int rows, int d, float eps,
                            int* zero, int n_zero, cudaStream_t stream, bool overlap) {
  (void)ctx;
  const int c8 = d / 8, kb = (d + 127) / 128;
  const int nv = (c8 + kThreads - 1) / kThreads;
  auto* xp = static_cast<const uint4*>(x);
  auto* qp = static_cast<uint2*>(q);
#define HB_QN(NV_)                                                                                              \
  if (nv <= NV_)                                                                                                \
    return launch(overlap, quant_norm_kernel<NV_>, rows, kThreads, 0, stream, "quant_norm_kernel launch", xp,   \
                  qp, scale, c8, kb, 1.0f / d, eps, zero, n_zero);
  HB_QN(1)
  HB_QN(2)
  HB_QN(4)
  HB_QN(8)
#undef HB_QN
  set_error("block-scaled layer: d_model = %d above the supported 16384", d);
  return HB_ERR_UNSUPPORTED;
}

hb_status quant_block_launch(const DeviceCtx& ctx, const void* x, void* q, float* scale, int rows, int cols,
                             int block_rows, cudaStream_t stream) {
  (void)ctx;
  const int c8 = cols / 8, kb = (cols + 127) / 128;
  auto* xp = static_cast<const uint4*>(x);
  auto* qp = static_cast<uint2*>(q);
  if (block_rows == 128)
    return launch_pdl(quant_blocks_kernel, dim3(kb, (rows + 127) / 128), kThreads, 0, stream,
                      "quant_blocks_kernel launch", xp, qp, scale, rows, c8, kb);
  int gshift = 0;
  while (gshift < 4 && (1 << gshift) < kb) ++gshift;
  const int rpc = 16 >> gshift;
  const int passes = (kb + (1 << gshift) - 1) >> gshift;
  const int gx = (rows + rpc - 1) / rpc;
#define HB_QG(U_)                                                                                              \
  return launch_pdl(quant_groups_kernel<U_>, dim3(gx, (passes + U_ - 1) / U_), kThreads, 0, stream,             \
                    "quant_groups_kernel launch", xp, qp, scale, rows, c8, kb, gshift)
  if (passes >= 4) HB_QG(4);
  if (passes >= 2) HB_QG(2);
  HB_QG(1);
#undef HB_QG
}

}  // namespace hb

extern "C" hb_status hb_quantize_e4m3_block(const void* x, void* q, float* scale, int32_t rows, int32_t cols,
                                            int32_t block_rows, void* stream) {
  hb::clear_error();
  HB_REQUIRE(rows == 0 || (x && q && scale), "hb_quantize_e4m3_block: null pointer");
  HB_REQUIRE(rows >= 0 && cols > 0 && cols % 16 == 0,
             "hb_quantize_e4m3_block: rows >= 0 and cols %% 16 == 0 required");
  HB_REQUIRE(block_rows == 1 || block_rows == 128, "hb_quantize_e4m3_block: block_rows must be 1 or 128, not %d",
             block_rows);
  HB_REQUIRE(cols <= hb::kMaxCols && rows <= hb::kMaxRows,
             "hb_quantize_e4m3_block: at most %d rows and %d columns", hb::kMaxRows, hb::kMaxCols);
  HB_REQUIRE(hb::aligned16(x) && hb::aligned16(q) && hb::aligned4(scale),
             "hb_quantize_e4m3_block: 16-byte alignment (scale: 4)");
  if (rows == 0) return HB_OK;
  hb::DeviceCtx ctx;
  hb_status st = hb::device_context(&ctx);
  if (st != HB_OK) return st;
  return hb::quant_block_launch(ctx, x, q, scale, rows, cols, block_rows, static_cast<cudaStream_t>(stream));
}
