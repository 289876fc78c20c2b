// index.cu -- write and read rows of the index-key cache.
//
// A key's 128 values become E2M1 codes with one E4M3 scale per 16 values
// (the encoding of the latent values in the NVFP4 row format of the Prime
// Inference post, section "Making room for low-latency decode"; the post
// takes the indexer's positions as given and does not describe its cache).
// Eight lanes hold a token, 16 values each: 32 bytes of bf16 in or out, 8
// bytes of codes, one scale byte; the eight scale bytes of a token go through
// one lane as one 8-byte word. HBM-bound for a chunk of tokens (256 + 72
// bytes each), launch-bound for a step of a few.
// Measured (GB300, device time): 66 tokens 2.5 us to write and 2.1 to read back;
// 32768 tokens 6.0 us (10.7 MB, 1.8 TB/s: the chain of block-table, key and row
// accesses of a single wave of CTAs) and 4.2 us (2.6 TB/s).
#include "index_common.cuh"

namespace nvfp4_mla {

bool index_shape_ok(int32_t num_seqs, int32_t max_blocks, int32_t page_size, int64_t num_blocks,
                    int64_t block_stride) {
  return num_seqs > 0 && max_blocks > 0 && page_size > 0 && page_size <= (1 << 20) &&
         page_size % 2 == 0 && num_blocks > 0 &&
         block_stride >= static_cast<int64_t>(page_size) * kIndexRow &&
         static_cast<int64_t>(num_seqs) * max_blocks <= (int64_t{1} << 40);
}

namespace {

constexpr int kIndexThreads = 256;
constexpr int kLanesPerTok = kIndexScales;  // 8
constexpr int kToksPerBlock = kIndexThreads / kLanesPerTok;

__global__ void __launch_bounds__(kIndexThreads)
    index_append_kernel(const uint8_t* __restrict__ keys, const int32_t* __restrict__ seq_ids,
                        const int32_t* __restrict__ positions, int32_t n_tok,
                        const int32_t* __restrict__ block_table, int32_t num_seqs,
                        int32_t max_blocks, int32_t page_size, uint8_t* __restrict__ cache,
                        int64_t num_blocks, int64_t block_stride,
                        int32_t* __restrict__ invalid_count) {
  const int part = threadIdx.x % kLanesPerTok;
  const int64_t t =
      static_cast<int64_t>(blockIdx.x) * kToksPerBlock + threadIdx.x / kLanesPerTok;
  const bool live = t < n_tok;
  uint32_t w[8] = {};
  int32_t seq = -1;
  IndexRow at = {-1, 0};
  if (live) {  // the key's loads overlap the index and block-table loads
    const uint8_t* src = keys + t * (kIndexDim * 2) + part * (kGroup * 2);
    const uint4 a = ld_nc_v4(src), b = ld_nc_v4(src + 16);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    seq = __ldg(seq_ids + t);
    at = resolve_index_row(seq, __ldg(positions + t), block_table, num_seqs, max_blocks,
                           page_size, num_blocks, block_stride);
  }
  uint32_t lo, hi;
  float scale;
  const uint32_t sc = quantize_group(w, lo, hi, scale);
  // the token's eight scale bytes, byte k from lane k
  uint64_t all = static_cast<uint64_t>(sc) << (8 * part);
#pragma unroll
  for (int d = 1; d < kLanesPerTok; d <<= 1) all |= __shfl_xor_sync(0xffffffffu, all, d);
  if (at.page < 0) {
    if (live && part == 0 && seq != -1 && invalid_count != nullptr) atomicAdd(invalid_count, 1);
    return;
  }
  uint8_t* page = cache + at.page;
  *reinterpret_cast<uint2*>(page + static_cast<int64_t>(at.row) * kIndexCodes + part * 8) =
      make_uint2(lo, hi);
  if (part == 0)
    *reinterpret_cast<uint64_t*>(page + static_cast<int64_t>(page_size) * kIndexCodes +
                                 static_cast<int64_t>(at.row) * kIndexScales) = all;
}

__global__ void __launch_bounds__(kIndexThreads)
    index_read_kernel(const int32_t* __restrict__ seq_ids, const int32_t* __restrict__ positions,
                      int32_t n_tok, const int32_t* __restrict__ block_table, int32_t num_seqs,
                      int32_t max_blocks, int32_t page_size, const uint8_t* __restrict__ cache,
                      int64_t num_blocks, int64_t block_stride, uint8_t* __restrict__ keys,
                      int32_t* __restrict__ invalid_count) {
  const int part = threadIdx.x % kLanesPerTok;
  const int64_t t =
      static_cast<int64_t>(blockIdx.x) * kToksPerBlock + threadIdx.x / kLanesPerTok;
  if (t >= n_tok) return;
  const int32_t seq = __ldg(seq_ids + t);
  const IndexRow at = resolve_index_row(seq, __ldg(positions + t), block_table, num_seqs,
                                        max_blocks, page_size, num_blocks, block_stride);
  uint32_t out[8] = {};
  if (at.page >= 0) {
    const uint8_t* page = cache + at.page;
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>(
        page + static_cast<int64_t>(at.row) * kIndexCodes + part * 8));
    const uint8_t sc = __ldg(page + static_cast<int64_t>(page_size) * kIndexCodes +
                             static_cast<int64_t>(at.row) * kIndexScales + part);
    const float s = f16_bits_to_f32(
        static_cast<uint16_t>(e4m3x2_to_f16x2(static_cast<uint16_t>(sc)) & 0xFFFFu));
    uint32_t h[8];
    {
      uint32_t a[4], b[4];
      e2m1x8_to_f16x8(codes.x, a);
      e2m1x8_to_f16x8(codes.y, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = a[i], h[4 + i] = b[i];
    }
    // a code has at most 2 significant bits and a scale 4: exact in bf16's 8
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[i] = pack_bf16x2(f16_bits_to_f32(static_cast<uint16_t>(h[i] & 0xFFFFu)) * s,
                           f16_bits_to_f32(static_cast<uint16_t>(h[i] >> 16)) * s);
  } else if (part == 0 && seq != -1 && invalid_count != nullptr) {
    atomicAdd(invalid_count, 1);
  }
  uint4* dst = reinterpret_cast<uint4*>(keys + t * (kIndexDim * 2) + part * (kGroup * 2));
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// Argument checks that both entry points share; OK and n_tok > 0: launch.
int32_t index_check(const void* keys, const int32_t* seq_ids, const int32_t* positions,
                    int32_t n_tok, const int32_t* block_table, int32_t num_seqs,
                    int32_t max_blocks, int32_t page_size, const void* cache, int64_t num_blocks,
                    int64_t block_stride) {
  if (!keys || !seq_ids || !positions || !block_table || !cache) return NVFP4_MLA_ERR_NULL;
  if (!index_shape_ok(num_seqs, max_blocks, page_size, num_blocks, block_stride))
    return NVFP4_MLA_ERR_SHAPE;
  if (!aligned16(keys) || !aligned16(cache) || (block_stride & 15)) return NVFP4_MLA_ERR_ALIGN;
  int dev = 0, sms = 0;
  return current_device_checked(&dev, &sms);
}

}  // namespace
}  // namespace nvfp4_mla

using namespace nvfp4_mla;

extern "C" int32_t nvfp4_mla_index_append(const void* keys, const int32_t* seq_ids,
                                          const int32_t* positions, int32_t n_tok,
                                          const int32_t* block_table, int32_t num_seqs,
                                          int32_t max_blocks_per_seq, int32_t page_size,
                                          void* cache, int64_t num_blocks,
                                          int64_t block_stride_bytes, int32_t* invalid_count,
                                          void* stream) {
  if (n_tok < 0) return NVFP4_MLA_ERR_SHAPE;
  if (n_tok == 0) return NVFP4_MLA_OK;
  if (int32_t st = index_check(keys, seq_ids, positions, n_tok, block_table, num_seqs,
                               max_blocks_per_seq, page_size, cache, num_blocks,
                               block_stride_bytes))
    return st;
  const unsigned grid = (static_cast<unsigned>(n_tok) + kToksPerBlock - 1) / kToksPerBlock;
  index_append_kernel<<<grid, kIndexThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(keys), seq_ids, positions, n_tok, block_table, num_seqs,
      max_blocks_per_seq, page_size, static_cast<uint8_t*>(cache), num_blocks,
      block_stride_bytes, invalid_count);
  return launch_status();
}

extern "C" int32_t nvfp4_mla_index_read(const int32_t* seq_ids, const int32_t* positions,
                                        int32_t n_tok, const int32_t* block_table,
                                        int32_t num_seqs, int32_t max_blocks_per_seq,
                                        int32_t page_size, const void* cache, int64_t num_blocks,
                                        int64_t block_stride_bytes, void* keys,
                                        int32_t* invalid_count, void* stream) {
  if (n_tok < 0) return NVFP4_MLA_ERR_SHAPE;
  if (n_tok == 0) return NVFP4_MLA_OK;
  if (int32_t st = index_check(keys, seq_ids, positions, n_tok, block_table, num_seqs,
                               max_blocks_per_seq, page_size, cache, num_blocks,
                               block_stride_bytes))
    return st;
  const unsigned grid = (static_cast<unsigned>(n_tok) + kToksPerBlock - 1) / kToksPerBlock;
  index_read_kernel<<<grid, kIndexThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      seq_ids, positions, n_tok, block_table, num_seqs, max_blocks_per_seq, page_size,
      static_cast<const uint8_t*>(cache), num_blocks, block_stride_bytes,
      static_cast<uint8_t*>(keys), invalid_count);
  return launch_status();
}
