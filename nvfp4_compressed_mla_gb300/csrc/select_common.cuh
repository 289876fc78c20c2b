// select_common.cuh -- what the two kernels of sparse_mla_select share.
//
// Kernel 1 writes fp32 scores (the highest of every `granule` = min(block, 32)
// consecutive positions) and, per tile of 128 positions, the largest scale
// byte among the keys; kernel 2 picks the blocks.
#pragma once

#include "index_common.cuh"

namespace nvfp4_mla {

constexpr int kScoreTile = 128;      // positions per tile of the score kernel
constexpr int kMaxGranule = 32;      // positions behind one stored score
constexpr int kStatusWords = 1024;   // one per CTA of the score kernel

struct SelectParams {
  const uint8_t* q_index;
  const float* weights;
  const int32_t* q_seq;
  const int32_t* q_pos;
  int32_t num_q, num_heads;
  const int32_t* block_table;
  int32_t num_seqs, max_blocks, page_size;
  const uint8_t* cache;
  int64_t num_blocks, block_stride;
  int32_t block, num_select, sink, recent;
  int32_t room;       // positions of a table's row: max_blocks * page_size
  int32_t take_all;   // num_select * block: up to here every visible position is taken
  int32_t* topk_idx;
  uint8_t* images;    // [num_q] images of the encoded queries
  float* scores;      // [num_q, score_stride]
  int64_t score_stride;
  // [num_q, tiles]: the largest key scale byte of each tile's quarters, in the
  // row of the first query token of a run (consecutive tokens of one sequence
  // inside an aligned group of `group`)
  uint32_t* smax;
  int64_t tiles;
  int32_t group;
  uint32_t* status;   // [kStatusWords]
  int32_t score_ctas;
  long long wait_cycles;
};

// Positions that a query token at `pos` of sequence `seq` sees, 0 for none.
__device__ __forceinline__ int32_t visible_positions(const SelectParams& p, int32_t seq,
                                                     int32_t pos) {
  return seq >= 0 && seq < p.num_seqs && pos >= 0 ? min(pos, p.room - 1) + 1 : 0;
}

// Positions that have to be scored: none where every visible block is taken.
__device__ __forceinline__ int32_t scored_positions(const SelectParams& p, int32_t seq,
                                                    int32_t pos) {
  const int32_t n = visible_positions(p, seq, pos);
  return n > p.take_all ? n : 0;
}

// Bytes of a query token's image.
size_t query_image_bytes(int32_t num_heads);

int32_t launch_scores(SelectParams& p, int num_sms, cudaStream_t stream);

}  // namespace nvfp4_mla
