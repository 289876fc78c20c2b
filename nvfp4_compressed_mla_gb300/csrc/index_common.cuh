// index_common.cuh -- the index-key cache: where a row lies in its page.
#pragma once

#include "common.cuh"

namespace nvfp4_mla {

constexpr int kIndexDim = NVFP4_MLA_INDEX_DIM;          // 128
constexpr int kIndexCodes = kIndexDim / 2;              // 64 bytes of codes per row
constexpr int kIndexScales = kIndexDim / kGroup;        // 8 scale bytes per row
constexpr int kIndexRow = NVFP4_MLA_INDEX_ROW_BYTES;    // 72
static_assert(kIndexCodes + kIndexScales == kIndexRow, "72-byte index row");

// A row's codes and scales are in two sections of its page.
struct IndexRow {
  int64_t page;  // byte offset of the page in the pool, -1: does not resolve
  int32_t row;
};

__device__ __forceinline__ IndexRow resolve_index_row(int32_t b, int32_t pos,
                                                      const int32_t* __restrict__ block_table,
                                                      int32_t num_seqs, int32_t max_blocks,
                                                      int32_t page_size, int64_t num_blocks,
                                                      int64_t block_stride) {
  if (b < 0 || b >= num_seqs || pos < 0) return {-1, 0};
  const int32_t lb = pos / page_size;
  if (lb >= max_blocks) return {-1, 0};
  const int64_t pb = __ldg(block_table + static_cast<int64_t>(b) * max_blocks + lb);
  if (pb < 0 || pb >= num_blocks) return {-1, 0};
  return {pb * block_stride, pos - lb * page_size};
}

// Scale byte of a group with the given largest magnitude, and its value.
__device__ __forceinline__ uint32_t group_scale(float amax, float& value) {
  // The fp32 quotient of a bf16 by 6 never sits on an E4M3 rounding midpoint
  // unless the exact quotient does, so this equals rounding the exact one.
  const uint32_t sc = cvt_e4m3x2(0.f, __fdiv_rn(amax, 6.0f)) & 0xFFu;
  value = f16_bits_to_f32(static_cast<uint16_t>(e4m3x2_to_f16x2(static_cast<uint16_t>(sc))));
  return sc;
}

// Codes of 16 bf16 values (8 words, two values each): element k in nibble k.
__device__ __forceinline__ uint32_t quantize_group(const uint32_t (&w)[8], uint32_t& lo,
                                                   uint32_t& hi, float& scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
  const uint32_t sc = group_scale(amax, scale);
  lo = hi = 0;
  if (scale > 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo |= e2m1_code(bf16_lo(w[i]), scale) << (8 * i) |
            e2m1_code(bf16_hi(w[i]), scale) << (8 * i + 4);
      hi |= e2m1_code(bf16_lo(w[4 + i]), scale) << (8 * i) |
            e2m1_code(bf16_hi(w[4 + i]), scale) << (8 * i + 4);
    }
  }
  return sc;
}

bool index_shape_ok(int32_t num_seqs, int32_t max_blocks, int32_t page_size, int64_t num_blocks,
                    int64_t block_stride);

}  // namespace nvfp4_mla
