// Pieces shared by the attention kernels over an E4M3 cache (attention_e4m3.cu:
// decode rows; attention_e4m3_chunk.cu: prompt chunks).
#pragma once
#include <cuda_bf16.h>

#include "device.cuh"
#include "runtime.h"

namespace hb {
namespace kv8 {

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
  __nv_bfloat16 *scratch_k, *scratch_v;  // widened sequences of several rows, [padded keys][d_head] a kv head
  int scratch_keys;                      // that it holds
  float* partials;  // split records [sequence][split][kv head]
  int max_splits;   // of a sequence of max_kv_len keys
  float* chunk_partials;  // records of chunk rows whose keys are split, [part_row][q head][part]
  int part_stride;        // rows of a sequence there; 0: by the plan's rows (part_row)
  int max_parts;          // of a sequence of max_kv_len keys
  int no_chunks;    // the plan has as many rows as sequences: none may have several
  // the plan has one sequence and more rows than that: the chunk kernel takes the
  // sequence even if it has one row (and the others of the plan are padding)
  int no_decodes;
  // 1 when the chunk kernel precedes the decode kernel on the stream: it waited
  // for the inputs before it let this one start, so the decode kernel's wait is
  // deferred to its end (whose completion then implies the chunk kernel's)
  int wait_at_end;
  int* status;
};

// A chunk of few rows has few units for the SMs, which take its keys block by
// block: they are split into as many parts as give kSplitUnits (an SM each), at
// most kMaxParts and of at least kPartBlocks blocks, joined afterwards.  By the
// sequence and the dims alone, so that a row's result does not depend on its
// batch; `blocks`: 128-key blocks that the first tile sees.
constexpr int kSplitUnits = 152, kMaxParts = 8, kPartBlocks = 8;
__host__ __device__ inline int part_count(int units, int blocks) {
  int n = blocks / kPartBlocks < kSplitUnits / units ? blocks / kPartBlocks : kSplitUnits / units;
  n = n < kMaxParts ? n : kMaxParts;
  return n < 1 ? 1 : n;
}
__host__ __device__ inline int first_tile_blocks(int qlen, int kvl) {
  return (kvl - qlen + (qlen < 128 ? qlen : 128) + 127) / 128;
}
// Most rows of a sequence whose keys are split: more have too many units.
inline int split_rows(int n_q) { return 128 * (kSplitUnits / 2 / n_q); }
// Which record row a row of sequence seq, which starts at q0, has: its place among
// the split_rows of its sequence, or its own number where the plan has fewer rows
// than that takes.
__device__ __forceinline__ int part_row(const Params& p, int row, int seq, int q0) {
  return p.part_stride > 0 ? seq * p.part_stride + row - q0 : row;
}
// a record: O [D], its maximum and sum, fp32 (a multiple of 16 bytes)
__host__ __device__ constexpr int part_floats(int d) { return d + 4; }

// E4M3 to bf16, exactly, two codes at a time, a code in the upper byte of each
// half: sign, and the exponent and mantissa fields moved to bf16's places make
// the value times 2^-120 (the exponents' biases differ by 120, and a subnormal
// code becomes a subnormal number); a product with 2^120 ends it.
__device__ __forceinline__ uint32_t codes_moved(uint32_t w) {
  return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace kv8

// Sequences of several rows: those that the scratch holds, widened into it and
// attended by `grid` CTAs; and those behind its end.
hb_status chunk_e4m3_launch(const DeviceCtx& ctx, const void* q, const kv8::Params& p, int d_head, int grid,
                            cudaStream_t stream);
hb_status chunk_e4m3_overflow_launch(const DeviceCtx& ctx, const void* q, const kv8::Params& p, int d_head,
                                     cudaStream_t stream);

}  // namespace hb
