// Residual addition, RMS norm and the projection operand in one pass.
//
//   h = bf16(x + residual)                  (h = x without a residual)
//   y = h / sqrt(mean(h^2) + eps) * gamma   (fp32, from the rounded h)
// with y stored as bf16, or as E4M3 codes with an fp32 scale per row or per
// 128 columns: inv = 448 / top, scale = top / 448 (correctly rounded), code =
// E4M3(fp32(y * inv)); a group of zeros gets scale 0 and zero codes.  top is
// amax |y|; of 128 columns 2^-112 at least, as in the block quantization.  A row's
// is taken as it is: where 448 / amax might not be finite, y and amax are first
// multiplied by 2^40.  y goes into its codes from fp32: the only
// roundings are h's to bf16, which is what the next residual reads, and the
// code's.
//
// Reads 4 and writes 3 or 4 bytes an element, each once: HBM bounds it for
// many rows, the chain load - sum - maximum - store for few.  8192 x 7168 with a
// scale per row: 61 us (floor 61.5 at the copy rate); one row of 4096 in blocks:
// 2.0 us.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace {

using namespace dev;

constexpr float kAmaxMin = 0x1p-112f;
constexpr float kLift = 0x1p40f;
constexpr int kMaxD = 32768;

struct NormArgs {
  const uint4 *x, *res, *gamma;
  uint4* h;
  void* y;
  float* scale;
  int rows, d8, kb;
  float inv_d, eps;
};

struct Scale {
  float inv, scale;
};
// of a maximum given as the bits of its magnitude (a NaN's are above all); of a row,
// inv is that of y and amax times `lift`
template <bool ROW>
__device__ __forceinline__ Scale scale_of(uint32_t amax, float lift) {
  if (amax == 0) return {0.f, 0.f};
  const float top = !ROW && amax < __float_as_uint(kAmaxMin) ? kAmaxMin : __uint_as_float(amax);
  return {__fdiv_rn(448.0f, ROW ? __fmul_rn(top, lift) : top), __fdiv_rn(top, 448.0f)};
}

__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[2 * j], inv), __fmul_rn(y[2 * j + 1], inv)), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// fp32 y of one 16-byte piece of h
__device__ __forceinline__ void normed(const uint4& h, const uint4& g, float inv, float (&y)[8]) {
  const uint32_t w[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_bf16x2(w[j]), gg = unpack_bf16x2(gw[j]);
    y[2 * j] = __fmul_rn(__fmul_rn(f.x, inv), gg.x);
    y[2 * j + 1] = __fmul_rn(__fmul_rn(f.y, inv), gg.y);
  }
}

__device__ __forceinline__ uint32_t magnitude(const float (&y)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7fffffffu);
  return m;
}

// TPR threads take a row (a warp, or the CTA) and hold it in registers: piece
// t + TPR k (16 bytes) is thread t's k-th, so the 16 pieces of 128 columns lie
// in 16 neighbouring lanes.  The sum of squares is formed in an order of the
// row length alone.
template <int NV, int FMT, int TPR>
__global__ void __launch_bounds__(256) add_rmsnorm_kernel(NormArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kWarps = TPR / 32;
  __shared__ float red[8];
  __shared__ uint32_t red_max[8];
  const int t = threadIdx.x % TPR;
  const int row = TPR == 256 ? blockIdx.x : blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (TPR < 256 && row >= a.rows) return;
  const size_t base = static_cast<size_t>(row) * a.d8;
  uint4 v[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = t + TPR * k;
    v[k] = i < a.d8 ? ld_u4(a.x + base + i) : make_uint4(0, 0, 0, 0);
  }
  if (a.res) {
    uint4 r[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = t + TPR * k;
      r[k] = i < a.d8 ? ld_u4(a.res + base + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, rw[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
      uint32_t s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack_bf16x2(w[j]), g = unpack_bf16x2(rw[j]);
        s[j] = pack_bf16x2(__fadd_rn(f.x, g.x), __fadd_rn(f.y, g.y));
      }
      v[k] = make_uint4(s[0], s[1], s[2], s[3]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = t + TPR * k;
    if (a.h && i < a.d8) a.h[base + i] = v[k];
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_bf16x2(w[j]);
      ss = __fmaf_rn(f.x, f.x, ss);
      ss = __fmaf_rn(f.y, f.y, ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
  if (kWarps > 1) {
    if ((t & 31) == 0) red[t >> 5] = ss;
    __syncthreads();
    ss = red[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) ss = __fadd_rn(ss, red[w]);
  }
  const float inv = rsqrtf(__fmaf_rn(ss, a.inv_d, a.eps));
  if (FMT == HB_NORM_BF16) {
    uint4* y = static_cast<uint4*>(a.y) + base;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = t + TPR * k;
      if (i >= a.d8) break;
      float f[8];
      normed(v[k], ld_u4(a.gamma + i), inv, f);
      y[i] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
    }
  } else if (FMT == HB_NORM_E4M3_BLOCK) {
    uint2* y = static_cast<uint2*>(a.y) + base;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = t + TPR * k;
      float f[8] = {};
      if (i < a.d8) normed(v[k], ld_u4(a.gamma + i), inv, f);
      uint32_t m = magnitude(f);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (i < a.d8) {
        const Scale s = scale_of<false>(m, 1.f);
        y[i] = codes8(f, s.inv);
        if ((t & 15) == 0) a.scale[static_cast<size_t>(row) * a.kb + i / 16] = s.scale;
      }
    }
  } else {
    uint2* y = static_cast<uint2*>(a.y) + base;
    uint4 g[NV];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = t + TPR * k;
      g[k] = i < a.d8 ? ld_u4(a.gamma + i) : make_uint4(0, 0, 0, 0);
      float f[8];
      normed(v[k], g[k], inv, f);
      // past the row's end h = 0 (where the row is NaN its own pieces say so)
      if (i < a.d8) m = max(m, magnitude(f));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (kWarps > 1) {
      if ((t & 31) == 0) red_max[t >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = max(m, red_max[w]);
    }
    const bool tiny = m < __float_as_uint(kAmaxMin);  // of the row: all its threads agree
    const Scale s = scale_of<true>(m, tiny ? kLift : 1.f);
    if (t == 0) a.scale[row] = s.scale;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = t + TPR * k;
      if (i >= a.d8) break;
      float f[8];
      normed(v[k], g[k], inv, f);
      if (tiny) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], kLift);
      }
      y[i] = codes8(f, s.inv);
    }
  }
}

template <int NV, int TPR>
hb_status add_rmsnorm_launch(const NormArgs& a, int fmt, cudaStream_t stream) {
  auto kernel = fmt == HB_NORM_BF16   ? add_rmsnorm_kernel<NV, HB_NORM_BF16, TPR>
                : fmt == HB_NORM_E4M3 ? add_rmsnorm_kernel<NV, HB_NORM_E4M3, TPR>
                                      : add_rmsnorm_kernel<NV, HB_NORM_E4M3_BLOCK, TPR>;
  constexpr int kRows = 256 / TPR;
  return launch_pdl(kernel, (a.rows + kRows - 1) / kRows, 256, 0, stream, "add_rmsnorm_kernel launch", a);
}

}  // namespace
}  // namespace hb

extern "C" hb_status hb_add_rmsnorm(const void* x, const void* residual, const void* gamma, void* h_out, void* y,
                                    float* y_scale, int32_t rows, int32_t d, float eps, int32_t format, void* stream) {
  using namespace hb;
  clear_error();
  HB_REQUIRE(format == HB_NORM_BF16 || format == HB_NORM_E4M3 || format == HB_NORM_E4M3_BLOCK,
             "hb_add_rmsnorm: unknown format %d", format);
  HB_REQUIRE(rows >= 0 && d > 0 && d % (format == HB_NORM_BF16 ? 8 : 16) == 0 && d <= kMaxD,
             "hb_add_rmsnorm: rows >= 0, d a multiple of %d and at most %d required", format == HB_NORM_BF16 ? 8 : 16,
             kMaxD);
  HB_REQUIRE(eps >= 0.f, "hb_add_rmsnorm: eps must be >= 0");
  if (rows == 0) return HB_OK;
  HB_REQUIRE(x && gamma && y, "hb_add_rmsnorm: null pointer");
  HB_REQUIRE((format == HB_NORM_BF16) == (y_scale == nullptr),
             "hb_add_rmsnorm: scales go with codes, and with codes only");
  HB_REQUIRE(aligned16(x) && aligned16(residual) && aligned16(gamma) && aligned16(h_out) && aligned16(y) &&
                 aligned4(y_scale),
             "hb_add_rmsnorm: 16-byte alignment (y_scale: 4)");
  DeviceCtx ctx;
  hb_status st = device_context(&ctx);
  if (st != HB_OK) return st;
  NormArgs a;
  a.x = static_cast<const uint4*>(x);
  a.res = static_cast<const uint4*>(residual);
  a.gamma = static_cast<const uint4*>(gamma);
  a.h = static_cast<uint4*>(h_out);
  a.y = y;
  a.scale = y_scale;
  a.rows = rows;
  a.d8 = d / 8;
  a.kb = (d + 127) / 128;
  a.inv_d = 1.0f / d;
  a.eps = eps;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // A warp a row up to 1024 columns (4 pieces a lane), the CTA above, whatever the
  // rows, so that a row's sum has one order.  Measured, 57344 rows of 1024, bf16 /
  // scale per row / per block: a warp 68 / 60 / 61 us, the CTA 78 / 101 / 90 (one
  // row: 2.0 / 2.0 / 2.8 and 1.5 / 1.7 / 1.6); 28672 rows of 2048: a warp 69 / 60 /
  // 71, the CTA 67 / 66 / 65, and one row 3.0 / 2.6 / 4.6 against 1.6 / 1.8 / 1.7.
  if (a.d8 <= 32) return add_rmsnorm_launch<1, 32>(a, format, s);
  if (a.d8 <= 64) return add_rmsnorm_launch<2, 32>(a, format, s);
  if (a.d8 <= 128) return add_rmsnorm_launch<4, 32>(a, format, s);
  if (a.d8 <= 256) return add_rmsnorm_launch<1, 256>(a, format, s);
  if (a.d8 <= 512) return add_rmsnorm_launch<2, 256>(a, format, s);
  if (a.d8 <= 1024) return add_rmsnorm_launch<4, 256>(a, format, s);
  if (a.d8 <= 2048) return add_rmsnorm_launch<8, 256>(a, format, s);
  return add_rmsnorm_launch<16, 256>(a, format, s);
}
