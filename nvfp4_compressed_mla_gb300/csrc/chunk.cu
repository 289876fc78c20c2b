// chunk.cu -- dense causal absorbed-MLA attention of a step's new tokens over the paged cache.
//
// Token i of the n new tokens of a sequence of length L sees keys 0 .. L - n + i. For each head
//   z_j = sm_scale (ql . lat_j + qr . rope_j),  out = sum_j softmax(z)_j lat_j,
// so keys and values are one row of the cache that all heads and tokens share: with M = (token,
// head) rows the step is two matrix products, S = Q K^T (576 deep) and O = P V (512 wide), with
// 2 x 1088 flop a row and key. A cache row of 352 bytes serves 128 heads with 279 kflop a token,
// 791 flop a byte: tensor-bound from one token of 128 heads on.
//
// The rows (token, head) of a sequence are consecutive in memory, and a row tile takes 256 of
// them, whatever the number of heads. One cluster of four CTAs works on a tile. 512 columns of fp32
// output for 128 rows are all of an SM's tensor memory, so that the two products live on different
// SMs, each as one MMA over a pair of them (cta_group::2, M = 256): an SM expands half of the keys,
// or half of the dimensions, and the pair shares them, which halves the work of expanding a key for
// a row. On one SM with 64 keys at a time an MMA whose A operand is in tensor memory takes as long
// as one with 128 (70 cycles), so that sequences of up to 128 rows gain nothing from M = 128.
//
//   score CTAs (ranks 0, 1): 128 rows each. Q stays in tensor memory (latent part, 256 columns, the
//     MMA's A operand) and shared memory (rope part). Eight warps expand 64 keys a CTA and key tile
//     (128 keys) into FP16 (exact: a code times its scale has 6 significant bits) in shared memory;
//     S of 128 keys goes into one of two buffers. Three groups of four softmax warps (thread = row)
//     take its pieces of 64 keys in turn, make P = 2^(s c - m) of them against a lazy reference m,
//     in FP16, and a warp copies it into the output CTA of the same rows.
//   output CTAs (ranks 2, 3): O (128 rows x 512, fp32) in tensor memory. Eight warps expand the
//     keys' latent part, each CTA 256 of the dimensions; twelve warps rescale O when a row's
//     reference moved, and write the output.
//   In both a warp loads the cache's rows and a warp issues the MMAs; the issuing warp of a pair's
//     second CTA tells the leader's what its CTA has ready.
//
// Work is dealt out in key tiles: a planning kernel lists the row tiles of the step with the key
// tiles that each sees, and every cluster (36 of them fit the device's 152 SMs) takes an equal,
// contiguous share of all of them. A row tile that is cut by the shares' borders is merged by a last
// kernel from fp32 partial results. Which row is cut, and so a result's last bits, depends on the
// whole step, but on nothing outside of it: the same arguments give the same bits.
//
// Measured (bf16 output, one call of the three kernels behind the other; a device's bf16 product of
// two large matrices: 1906 TFLOP/s at best, 1709 for seconds on end; the first two by the power left):
//   NVFP4, 512 tokens of a prompt of 16384, 128 heads      1.24 - 1.31 ms  1760 - 1855 TFLOP/s
//   FP8, the same                                          1.26 - 1.30 ms  1770 - 1820
//   NVFP4, 5 prompts of up to 5000 tokens, 32 heads        1.12 ms  1560
//   FP8, the same                                          1.15 ms  1525
//   NVFP4, 61 sequences: prompts, drafts, single tokens    3.63 ms  1690 (6.1 PFLOP; others by their pairing)
//   NVFP4, 66 tokens of 66 contexts of up to 32768         0.50 ms   903 (half of each MMA's rows are empty)
//   FP8, the same                                          0.56 ms   800
//   NVFP4, the same with 8 / 32 / 64 heads                 0.48 / 0.49 / 0.49 ms
//   the same with pages of 16, 32 or 48 tokens             1.86 - 1.89 ms; the prompt above 4.59
//   NVFP4, 1 token of 128 heads, 8192 keys                   37 us  (bound by latency)
//   NVFP4, 7 tokens of 16 heads, 307 keys                    28 us
// The prompts are bound by the MMAs (the score SMs' tensor cores are active 95 % of the cycles). With a
// third of the MMAs the same pipelines (rows, expansion, softmax) took 1.13 and 1.19 ms for the first
// two, the 66 tokens 0.46: an MMA of 128 rows would not help those much. They do not depend on the
// rows either, so that fewer heads gain nothing. What a row tile
// costs beside its key tiles is loading Q and the first tile before P V can begin (8 us, most of it
// beside the tile before) and writing O (2.6 us). A short call is a chain: plan 3.7 us, rows and Q 5, first scores
// 2.5, first weights 3, a key tile 1.2 us each, output 2 to 4.5, teardown 2, merge 4 to 9.
// Pages that are no multiple of 64 tokens are copied row by row, 64 small copies in place of one, behind
// a lookup of the table that waits for a free slot.
//
// Every wait is bounded. A cluster whose wait runs out drains what it has in flight and reports
// it; the last kernel then writes NaN to all rows of the step.
#include <cuda.h>
#include <float.h>
#include <math.h>

#include <atomic>

#include "decode_common.cuh"
#include "plan_common.cuh"
#include "tc_ptx.cuh"

namespace nvfp4_mla {
namespace {

constexpr int kTileRows = 256, kTileKeys = 128;
constexpr int kPieceKeys = 64;                // keys of a P piece and of a V slot
constexpr uint32_t kGroups = 3;               // of four warps: softmax / rescaling and output
constexpr int kSoftWarps = 4 * kGroups;
constexpr int kExpandWarp0 = kSoftWarps, kExpandWarps = 8;
constexpr int kIssueWarp = kExpandWarp0 + kExpandWarps, kSendWarp = kIssueWarp + 1, kLoadWarp = kIssueWarp + 2;
constexpr int kChunkThreads = (kIssueWarp + 4) * 32;  // the last four warps leave registers to the others
// Registers of a thread of the softmax, the expanding and the last warps; as
// many in all as at the launch.
constexpr int kLaunchRegs = 80, kSoftRegs = 104, kExpandRegs = 64, kIssueRegs = 40;
static_assert(kGroups * kSoftRegs + 2 * kExpandRegs + kIssueRegs == 6 * kLaunchRegs, "registers");
constexpr int kMaxClusters = 40;
constexpr uint32_t kPBytes = 128 * kPieceKeys * 2;
constexpr uint32_t kKBlock = kPieceKeys * 128;   // 64 keys x 64 dimensions, FP16
constexpr uint32_t kTileBlocks = 9;              // 8 latent blocks and the rope
constexpr uint32_t kVSlotBytes = 4 * kKBlock;    // 64 keys x 256 dimensions
constexpr long long kDrainLimit = 1ll << 31;
// The reference of a row moves when a score exceeds it by more than kTau (log2
// units), to kHeadroom below that score. P <= 2^15 fits FP16 (largest finite
// value 65504) and P of the largest score is at least 2^kHeadroom then, so that
// weights down to 2^-16 of it are normal FP16 numbers and smaller ones are off by
// 2^-27 of it at most. A move stops the pipeline for an O in tensor memory to be
// read and written, so that room for scores to grow is worth more than precision
// of small weights: with kHeadroom 7 a third of the pieces had one.
constexpr float kTau = 15.f, kHeadroom = 2.f;
// Key tiles' time that a row tile costs beside its own (loading Q, the first
// score tile before P V can begin, writing O). With 1 / 2 / 3 / 4 / 5 key tiles
// five prompts of 5000 tokens take 1312 / 1241 / 1195 / 1155 / 1152 us (FP8 rows)
// and 61 sequences of all kinds 3730 / 3670 / 3617 / 3613 / 3626.
// The least share of a cluster is that overhead: a cluster more costs its start
// and a merge (4 us), a key tile 1.2 us. In a graph, a token of 128 heads over 384 /
// 768 / 2048 / 8192 keys takes 24.2 / 28.6 / 29.5 / 32.4 us with a least share of 4;
// 26.0 / 27.8 / 28.5 / 33.6 with 3, 23.8 / 27.0 / 32.3 / 34.1 with 7, 23.7 / 28.2 / 33.5 /
// 36.9 with 8. Over 97 short steps (1 to 32 sequences of 128 to 16384 tokens, 1 to
// 20 new ones) 3 is 0.5 % below 4 in the mean (9 % above and below it at the ends),
// 7 is 3 % above 4, 8 is 6 % and 12 is 11 %.
constexpr int kTileOverhead = 4, kLeastShare = kTileOverhead;

struct alignas(16) RowTile {  // 256 rows of a sequence
  int32_t seq, rows;     // its rows, 1 .. 256
  int32_t base, len;     // tokens before the new ones; length
  int64_t unit, end;     // its units: kTileOverhead, then one a key tile
  int64_t row0;          // its first row of all
  int32_t offset, pad;   // and of the sequence's
};
struct Plan {
  int64_t units, share;  // of all row tiles, of a cluster
  int32_t tiles, pad;
};

struct ChunkParams {
  const uint16_t* q_lat;
  const uint16_t* q_rope;
  const int32_t* cu_tokens;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t num_q, num_heads, num_seqs, max_blocks;
  PageSize page;
  const uint8_t* cache;
  int64_t num_blocks, block_stride;
  float score_scale;  // |sm_scale| log2(e), times latent_scale for FP8 rows
  float lat_mult;     // of Q's latent part: the sign of sm_scale
  float rope_mult;    // of its rope part: sign, and rope_scale (/ latent_scale)
  float out_mult;     // latent_scale for FP8 rows, else 1
  void* out;
  int32_t out_fp32;
  float* lse;
  int32_t* invalid_count;
  // workspace
  Plan* plan;
  RowTile* tiles;     // [max_tiles]
  int32_t* first;     // [clusters] the row tile of a cluster's first unit
  int32_t* failed;    // [clusters]
  float* part_lse;    // [2 clusters][rows]
  float* part_out;    // [2 clusters][rows][512]
  int32_t clusters, max_tiles;
  long long wait_cycles;
};

// Number of new tokens of sequence s and its length; 0 tokens for a malformed one.
__device__ __forceinline__ int32_t new_tokens(const ChunkParams& p, int32_t s, int32_t& start,
                                              int32_t& len) {
  start = __ldg(p.cu_tokens + s);
  const int32_t end = __ldg(p.cu_tokens + s + 1);
  len = __ldg(p.seq_lens + s);
  if (start < 0 || end < start || end > p.num_q || len < end - start ||
      len > static_cast<int64_t>(p.max_blocks) * p.page.size)
    return 0;
  return end - start;
}

// ------------------------------------------------------------------ planning
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p) {
  extern __shared__ int32_t upto[];  // [num_seqs] row tiles up to and with sequence s
  __shared__ int64_t sums[32];
  cudaTriggerProgrammaticLaunchCompletion();
  const int tid = threadIdx.x;
  int64_t tiles = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int32_t start, len;
    const int64_t rows =
        s < p.num_seqs ? static_cast<int64_t>(new_tokens(p, s, start, len)) * p.num_heads : 0;
    const int64_t to = block_scan((rows + kTileRows - 1) / kTileRows, tiles, sums);
    // offsets that overlap could ask for more than there is room for
    if (s < p.num_seqs) upto[s] = static_cast<int32_t>(min(to, static_cast<int64_t>(p.max_tiles)));
  }
  const int32_t n_tiles = static_cast<int32_t>(min(tiles, static_cast<int64_t>(p.max_tiles)));
  __syncthreads();
  int64_t units = 0;
  for (int t0 = 0; t0 < n_tiles; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int64_t n = 0;
    int s = 0;
    RowTile tile = {};
    if (t < n_tiles) {
      int hi = p.num_seqs - 1;
      while (s < hi) {
        const int mid = (s + hi) >> 1;
        if (upto[mid] <= t) s = mid + 1;
        else hi = mid;
      }
      const int64_t offset = static_cast<int64_t>(t - (s > 0 ? upto[s - 1] : 0)) * kTileRows;
      int32_t start, len;
      const int32_t tokens = new_tokens(p, s, start, len);
      const int64_t rows = min(static_cast<int64_t>(tokens) * p.num_heads - offset, int64_t{kTileRows});
      const int64_t last = (offset + rows - 1) / p.num_heads;  // token: it sees len - tokens + last + 1 keys
      n = kTileOverhead + (len - tokens + last + kTileKeys) / kTileKeys;
      tile = {s, static_cast<int32_t>(rows), len - tokens, len, 0, 0,
              static_cast<int64_t>(start) * p.num_heads + offset, static_cast<int32_t>(offset), 0};
    }
    const int64_t to = block_scan(n, units, sums);
    if (t < n_tiles) {
      tile.unit = to - n;
      tile.end = to;
      p.tiles[t] = tile;
    }
  }
  const int64_t share = max((units + p.clusters - 1) / p.clusters, int64_t{kLeastShare});
  // the row tile of each cluster's first unit
  for (int c = tid; c < p.clusters; c += kPlanThreads) {
    p.first[c] = n_tiles;
    p.failed[c] = 0;
  }
  if (tid == 0) *p.plan = {units, share, n_tiles, 0};
  __syncthreads();
  for (int t = tid; t < n_tiles; t += kPlanThreads) {
    const int64_t a = p.tiles[t].unit, b = p.tiles[t].end;
    for (int64_t c = (a + share - 1) / share; c * share < b; ++c) p.first[c] = t;
  }
}

// Adds n to a counter that stays at 2^31 - 1 where it would pass that.
__device__ __forceinline__ void add_saturating(int32_t* count, int64_t n) {
  int32_t was = *count;
  while (true) {
    const int32_t to = static_cast<int32_t>(min(was + n, int64_t{INT32_MAX}));
    const int32_t seen = atomicCAS(count, was, to);
    if (seen == was) return;
    was = seen;
  }
}

// Positions without a page, and malformed sequences; launched where they are counted.
__global__ void __launch_bounds__(256) chunk_check_kernel(const ChunkParams p) {
  __shared__ unsigned long long total;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  int64_t bad = 0;
  for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
    int32_t start, len;
    if (new_tokens(p, s, start, len) == 0) {
      const bool none = __ldg(p.cu_tokens + s) == __ldg(p.cu_tokens + s + 1);
      if (threadIdx.x == 0 && !none) ++bad;
      continue;
    }
    const int32_t blocks = p.page.blocks(len);
    for (int32_t b = threadIdx.x; b < blocks; b += 256) {
      const int32_t page = __ldg(p.block_table + static_cast<int64_t>(s) * p.max_blocks + b);
      if (page < 0 || page >= p.num_blocks) bad += min(p.page.size, len - b * p.page.size);
    }
  }
  if (bad > 0) atomicAdd(&total, static_cast<unsigned long long>(bad));
  __syncthreads();
  if (threadIdx.x == 0 && total > 0) add_saturating(p.invalid_count, static_cast<int64_t>(total));
}

// The pieces of row tiles that make up a cluster's share, one after the other. The
// plan is read through L1: the warps of a CTA follow one another through it.
struct Pieces {
  const ChunkParams& p;
  int64_t u0, u1;     // the cluster's units
  int32_t t, tiles;   // the next row tile
  int32_t cluster;
  // the current piece
  RowTile tile;
  int32_t begin, end;  // key tiles
  bool whole;          // all that the row tile sees
  int32_t slot;        // of a partial result

  __device__ Pieces(const ChunkParams& params, int c) : p(params), cluster(c) {
    const int64_t units = p.plan->units, share = p.plan->share;
    u0 = c * share;
    u1 = min(u0 + share, units);
    tiles = p.plan->tiles;
    t = u0 < units ? p.first[c] : tiles;
  }
  __device__ __forceinline__ bool next() {
    while (t < tiles) {
      tile = p.tiles[t];
      if (tile.unit >= u1) break;
      ++t;
      const int64_t k0 = tile.unit + kTileOverhead;  // unit of key tile 0
      begin = static_cast<int32_t>(max(u0 - k0, int64_t{0}));
      end = static_cast<int32_t>(max(min(u1, tile.end) - k0, int64_t{0}));
      if (end <= begin) continue;
      whole = begin == 0 && end == tile.end - k0;
      slot = 2 * cluster + (tile.unit >= u0 ? 1 : 0);
      return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------ PTX
// shared (this CTA) -> shared (another CTA of the cluster), counted on that CTA's mbarrier
__device__ __forceinline__ void bulk_s2s(uint32_t dst_cluster, uint32_t src, uint32_t bytes,
                                         uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst_cluster),
      "r"(src), "r"(bytes), "r"(bar_cluster)
      : "memory");
}
// An arrival at another CTA's barrier. What it reports lies in this CTA's own
// memories, where the tensor core of this SM reads it, and this thread has seen it
// complete; so release at CTA scope is enough. At cluster scope the arrival takes
// about 1000 cycles.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void st_relaxed_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_relaxed_cluster(uint32_t addr) {  // of this CTA's memory
  uint32_t v;
  asm volatile("ld.relaxed.cluster.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {  // multiples of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
template <int kRegs>
__device__ __forceinline__ void set_registers() {  // of all warps of a warpgroup
  if constexpr (kRegs > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
__device__ __forceinline__ void alloc_tmem_pair(uint32_t dst_smem) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(kTmemCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void free_tmem_pair(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kTmemCols)
               : "memory");
}
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrival on the barrier at this offset in every CTA of `mask`, once all
// MMAs that this thread issued before have completed.
__device__ __forceinline__ void commit_to(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle, 8-row groups 1024 bytes
// apart; `lead` is the distance of 64-element blocks along N (MN-major only).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead = 16) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
// Byte offset of 16-byte column `col` (0..7) of row `row` in a block of 128-byte rows.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t col) {
  return row * 128u + ((col ^ (row & 7u)) << 4);
}
// A bounded wait of a whole warp: every lane tests (and so acquires), and the lanes
// leave together with one result. The votes stand where the warp is converged:
// behind a loop of each lane's own they cost the kernel 7 %.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort_addr,
                                          long long limit) {
  if (__all_sync(0xffffffffu, mbar_test<kCluster>(bar, parity))) return true;
  const long long t0 = clock64();
  const uint32_t hint = suspend_ns(limit);
  while (true) {
    if (__all_sync(0xffffffffu, mbar_wait_suspend<kCluster>(bar, parity, hint))) return true;
    const bool late = clock64() - t0 > limit;
    if (__any_sync(0xffffffffu, late || ld_shared_u32(abort_addr) != 0u)) {
      if (late) st_shared_u32(abort_addr, 1u);
      return false;
    }
  }
}
// The same for a word of another CTA to become that of a tile; `word` is what was read last.
__device__ __forceinline__ bool warp_wait_word(uint32_t addr, uint32_t tile, uint32_t& word, uint32_t abort_addr,
                                               long long limit) {
  if (__all_sync(0xffffffffu, (word >> 1) == tile + 1)) return true;
  const long long t0 = clock64();
  while (true) {
    word = ld_relaxed_cluster(addr);
    if (__all_sync(0xffffffffu, (word >> 1) == tile + 1)) return true;
    const bool late = clock64() - t0 > limit;
    if (__any_sync(0xffffffffu, late || ld_shared_u32(abort_addr) != 0u)) {
      if (late) st_shared_u32(abort_addr, 1u);
      return false;
    }
  }
}
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_test<true>(bar, parity) && clock64() - t0 < kDrainLimit) {
  }
}
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {  // of a NaN and a number: the number
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t to_f16x2(uint32_t x, float m) {  // 2 bf16 values times m
  return pack_f16x2(bf16_lo(x) * m, bf16_hi(x) * m);
}
// Two pieces of 16 bytes, 64 bytes apart.
__device__ __forceinline__ void ld_two_v4(const uint16_t* p, uint32_t (&v)[8]) {
  const uint4 a = ld_nc_v4(p), b = ld_nc_v4(p + 32);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// The same lanes' 64 columns the other way.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 " NVFP4_TMEM_REGS ", [%32];"
               : NVFP4_TMEM_OUTS(r)
               : "r"(taddr)
               : "memory");
}
// Sixteen lanes of tensor memory, 32 columns: of a thread, registers 4 j + {0, 1}
// are columns 8 j + 2 (lane % 4) + {0, 1} of row lane / 4, and 4 j + {2, 3} of row lane / 4 + 8.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ------------------------------------------------------------------ memory plan
template <int kFmt>
struct ChunkLayout {
  static constexpr bool kNv = kFmt == NVFP4_MLA_ROW_NVFP4_352;
  static constexpr uint32_t kRow = kNv ? kNvfp4Row : kFp8Row;
  static constexpr uint32_t kRawBytes = kPieceKeys * kRow;  // cache rows of 64 keys
  // score CTA
  // A ring of blocks of keys. Two whole tiles of them would leave no room for what else
  // is worth more: two slots of NVFP4 rows on their way, two stages of P beside the one
  // slot of FP8 rows. So a tile's first kKBlocks - 9 blocks have room beside the tile
  // before, the others where the MMAs are done with that one's first ones. Of 512 tokens
  // of a prompt of 16384 (128 heads) and 66 single tokens over up to 32768 keys:
  // NVFP4 rows 1243 and 499 us with 15 blocks and two slots of rows, 1323 and 526 with 14
  // and two, 1248 and 543 with 16 and one. FP8 rows 1287 and 561 us with 16 blocks and two
  // stages, 1336 and 568 with 14 and two, 1319 and 570 with 14 and three.
  static constexpr uint32_t kK = 0, kKBlocks = kNv ? kTileBlocks + 6 : kTileBlocks + 7;
  static constexpr uint32_t kKShared = 2 * kTileBlocks - kKBlocks;  // blocks that wait for the tile before
  static_assert(kKBlocks >= kTileBlocks + 4 && kKShared > 0, "the expanding warps write four blocks at first");
  static constexpr uint32_t kQRope = kKBlocks * kKBlock;
  static constexpr uint32_t kStages = 2;                   // P pieces on their way out
  static constexpr uint32_t kStaged = kQRope + 16384;
  static constexpr uint32_t kRawScore = kStaged + kStages * kPBytes;
  static constexpr uint32_t kRawsScore = kNv ? 2 : 1;
  static constexpr uint32_t kRef = kRawScore + kRawsScore * kRawBytes;  // references of the rows, a group
  static constexpr uint32_t kSums = kRef + kGroups * 512;               // sums of weights, a group and 4 results
  static constexpr uint32_t kEndScore = kSums + 4 * kGroups * 512;
  // output CTA
  static constexpr uint32_t kVSlots = 3, kPSlots = kNv ? 4 : 3;
  static constexpr uint32_t kV = 0;
  static constexpr uint32_t kP = kV + kVSlots * kVSlotBytes;
  static constexpr uint32_t kRawOut = kP + kPSlots * kPBytes;
  static constexpr uint32_t kRawsOut = 2;
  // what may come with a piece: rescale factors of the rows, 1 + the piece for
  // each 32 of them that it is for; output factors of the rows, a result
  static constexpr uint32_t kNotes = 8;  // pieces (results) that may be noted and not yet done
  static constexpr uint32_t kFactor = kRawOut + kRawsOut * kRawBytes;
  static constexpr uint32_t kTag = kFactor + kNotes * 512;
  static constexpr uint32_t kFinal = kTag + kNotes * 16;
  static constexpr uint32_t kEndOut = kFinal + kNotes * 512;
  // a piece is noted once its stage is free: those that are staged or have a slot
  static_assert(kNotes > kPSlots + kStages, "notes");
  static constexpr uint32_t kCtl = kEndScore > kEndOut ? kEndScore : kEndOut;
  static constexpr uint32_t kCtlBytes = 1104;
  static constexpr uint32_t kBytes = kCtl + kCtlBytes;
  static_assert(kBytes <= kMaxSharedBytes && kCtl % 16 == 0 && kTag % 16 == 0, "shared memory");
  static_assert(kStaged % 1024 == 0 && kP % 1024 == 0 && kRawScore % 16 == 0 && kRawOut % 16 == 0, "operands");
};
constexpr uint32_t kSCol = 256;  // score CTA's tensor memory: Q's latent part, then two tiles of S
static_assert(kSCol + 2 * kTileKeys <= kTmemCols, "tensor memory");
struct ChunkCtl {  // barriers and words, at the same offsets in every CTA of the cluster
  static constexpr uint32_t kRawFull = 0, kRawEmpty = 16, kKFull = 32, kPeer = 48, kSFull = 64, kSEmpty = 80,
                            kQFull = 96, kStaged = 104, kStageFree = 128, kRefDone = 160, kSumDone = 256,
                            kPFull = 640, kPReady = 672, kPvDone = 704, kVFull = 736, kTask = 760,
                            kTaskDone = 768, kKHalf = 776, kTmem = 792, kAbort = 796, kSent = 800,
                            kScored = 804, kSummed = 808, kLoaded = 812, kTaskWord = 816, kNoted = 820,
                            kMissing = 848;
  // A CTA of the pair and 8 tiles: 2 (1 + tile), + 1 where one of its 64 keys has no page,
  // and then the bits of those that have one. The loader of the CTA writes it into both,
  // and no barrier says that it has arrived: whoever reads the word waits for its tile's.
  static constexpr uint32_t kMissingTiles = 8;
};
static_assert(ChunkCtl::kMissing + 32 * ChunkCtl::kMissingTiles == ChunkLayout<0>::kCtlBytes, "control block");
// The loader has the place of tile u - kMissingTiles for tile u: the expanding warps have left the rows
// of tile u - raws, so the MMAs of tile u - raws - 3 are done, and for those both CTAs' softmax warps
// have read the scores, and before them the word, of tile u - raws - 5.
static_assert(ChunkCtl::kMissingTiles >= ChunkLayout<0>::kRawsScore + 5 &&
                  ChunkCtl::kMissingTiles >= ChunkLayout<1>::kRawsScore + 5,
              "missing keys");

// ------------------------------------------------------------------ expansion
// Warp w of the eight expands keys 8 w .. 8 w + 7 of each 64; of the rope part a lane
// has 16 values of key lane / 4. Shared memory carries these reads and stores, the
// MMAs' operands and the copies of rows and P at once, so that no eight lanes' 16-byte
// accesses may meet in a bank: with FP8 rows read as a key a lane (four meet) 512
// tokens of a prompt took 1553 us in place of 1300.
//
// What the matrix products call a dimension need not be the row's. Within each
// block of 64 the order is such that what four lanes load of a row of Q, or write
// of O, with one 16-byte access each through the 16 x 256 bit shape of tensor
// memory is contiguous in global memory (q = 0 .. 3 is lane % 4 there):
//   keys (and Q): dimension 32 h + 8 q + 4 j + e is at 32 h + 16 j + 4 q + e  (h, j = 0, 1; e = 0 .. 3)
//   values (and O): dimension 32 h + 8 q + 2 j + e is at 32 h + 8 j + 2 q + e  (h, e = 0, 1; j = 0 .. 3)
// A score CTA expands all 512 dimensions of its keys, a CTA of the output pair
// dimensions 128 part .. + 127 of each half.
template <int kFmt, bool kKeys>
struct RowItems;

// 448, the largest E4M3 value, in place of a NaN.
__device__ __forceinline__ uint32_t as_number(uint32_t f) { return hmin2(f, 0x5F005F00u); }

template <bool kKeys>
struct RowItems<NVFP4_MLA_ROW_NVFP4_352, kKeys> {
  static constexpr uint32_t kRow = kNvfp4Row;
  static constexpr int kBlocks = kKeys ? 2 : 1;  // of a lane: lane / 8, and 4 more
  uint4 lat[kBlocks][2];
  uint32_t scale[kBlocks];
  uint4 rope;

  // A lane has key lane % 8 and blocks of 64 dimensions. Rows are 88 banks apart, so that keys 4 apart
  // meet in theirs: the later four lanes of eight read their halves the other way round.
  __device__ __forceinline__ void load(uint32_t raw, int w, int lane, uint32_t part) {
    const uint32_t key = raw + (8 * w + (lane & 7)) * kRow;
    const bool turned = (lane & 4) != 0;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const uint32_t b = (lane >> 3) + 4 * i;
      const uint32_t dim = kKeys ? 64 * b : 256 * (b >> 1) + 128 * part + 64 * (b & 1);
      const uint4 x = ld_shared_v4(key + dim / 2 + (turned ? 16 : 0));
      const uint4 y = ld_shared_v4(key + dim / 2 + (turned ? 0 : 16));
      lat[i][0] = turned ? y : x;
      lat[i][1] = turned ? x : y;
      scale[i] = ld_shared_u32(key + kScaleOff + dim / 16);
    }
    if constexpr (kKeys) rope = ld_shared_v4(raw + (8 * w + (lane >> 2)) * kRow + kRopeOff + 16 * (lane & 3));
  }

  // Blocks 4 i .. 4 i + 3 of the keys; at(block) is a block's 64 keys x 64 dimensions.
  template <typename At>
  __device__ __forceinline__ void store_blocks(int i, At&& at, int w, int lane) const {
    const uint32_t key = 8u * w + (lane & 7), block = at(4u * i + (lane >> 3));
    auto put = [&](uint32_t col, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      st_shared_v4(block + swizzled(key, col), a, b, c, d);
    };
    uint32_t s01 = e4m3x2_to_f16x2(static_cast<uint16_t>(scale[i] & 0xFFFFu));
    uint32_t s23 = e4m3x2_to_f16x2(static_cast<uint16_t>(scale[i] >> 16));
    if (!kKeys) {
      s01 = as_number(s01);
      s23 = as_number(s23);
    }
    const uint32_t s[4] = {__byte_perm(s01, s01, 0x1010), __byte_perm(s01, s01, 0x3232),
                           __byte_perm(s23, s23, 0x1010), __byte_perm(s23, s23, 0x3232)};
    const uint32_t words[8] = {lat[i][0].x, lat[i][0].y, lat[i][0].z, lat[i][0].w,
                               lat[i][1].x, lat[i][1].y, lat[i][1].z, lat[i][1].w};
    // the eight dimensions 32 h + 8 q .. + 7
    auto eight = [&](int h, int q, uint32_t (&f)[4]) {
      e2m1x8_to_f16x8(words[4 * h + q], f);
#pragma unroll
      for (int y = 0; y < 4; ++y) f[y] = hmul2_u32(f[y], s[2 * h + (q >> 1)]);
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kKeys) {
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          uint32_t f[4], g[4];
          eight(h, q, f);
          eight(h, q + 1, g);
          put(4 * h + (q >> 1), f[0], f[1], g[0], g[1]);
          put(4 * h + 2 + (q >> 1), f[2], f[3], g[2], g[3]);
        }
      } else {
        uint32_t f[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) eight(h, q, f[q]);
#pragma unroll
        for (int y = 0; y < 4; ++y) put(4 * h + y, f[0][y], f[1][y], f[2][y], f[3][y]);
      }
    }
  }
};

// A lane has half a block: 32 dimensions of key 4 (lane / 8 % 2) + 2 (lane / 4 % 2) +
// lane % 2, half lane / 2 % 2 of every second block. Rows are 144 banks apart, so that
// keys 2 apart meet in theirs: of eight lanes those with the later keys read their two
// 16 bytes the other way round, and neither their reads nor their stores conflict.
template <bool kKeys>
struct RowItems<NVFP4_MLA_ROW_FP8_576, kKeys> {
  static constexpr uint32_t kRow = kFp8Row;
  static constexpr int kItems = kKeys ? 4 : 2;
  uint4 lat[kItems][2];
  uint4 rope;

  static __device__ __forceinline__ uint32_t key_of(int w, int lane) {
    return 8u * w + ((lane >> 1) & 6) + (lane & 1);
  }
  __device__ __forceinline__ void load(uint32_t raw, int w, int lane, uint32_t part) {
    const uint32_t half = (lane >> 1) & 1, turned = (lane >> 2) & 1;
    const uint32_t from = raw + key_of(w, lane) * kRow + 32 * half;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const uint32_t b = (lane >> 4) + 2 * i;
      const uint32_t dim = kKeys ? 64 * b : 256 * (b >> 1) + 128 * part + 64 * (b & 1);
      const uint4 x = ld_shared_v4(from + dim + 16 * turned), y = ld_shared_v4(from + dim + 16 * (turned ^ 1));
      lat[i][0] = kKeys || turned == 0 ? x : y;
      lat[i][1] = kKeys || turned == 0 ? y : x;
    }
    if constexpr (kKeys) rope = ld_shared_v4(raw + (8 * w + (lane >> 2)) * kRow + kLatent + 16 * (lane & 3));
  }

  // Blocks 4 i .. 4 i + 3 of the keys; at(block) is a block's 64 keys x 64 dimensions.
  template <typename At>
  __device__ __forceinline__ void store_blocks(int i, At&& at, int w, int lane) const {
    const uint32_t key = key_of(w, lane), half = (lane >> 1) & 1, turned = (lane >> 2) & 1;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint4(&v)[2] = lat[2 * i + x];
      const uint32_t block = at(4u * i + 2 * x + (lane >> 4));
      // dimensions 16 z + 8 q + 2 y, + 1 of the half (of its turned parts, for keys)
      auto two = [&](int z, int q, int y) {
        const uint32_t word = q ? ((y >> 1) ? v[z].w : v[z].z) : ((y >> 1) ? v[z].y : v[z].x);
        const uint32_t f = e4m3x2_to_f16x2(static_cast<uint16_t>(word >> (16 * (y & 1))));
        return kKeys ? f : as_number(f);
      };
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if constexpr (kKeys) {
          const int z = m & 1, y = m & 2;
          st_shared_v4(block + swizzled(key, 4 * half + (z ^ turned) + y), two(z, 0, y), two(z, 0, y + 1),
                       two(z, 1, y), two(z, 1, y + 1));
        } else {
          st_shared_v4(block + swizzled(key, 4 * half + m), two(0, 0, m), two(0, 1, m), two(1, 0, m), two(1, 1, m));
        }
      }
    }
  }
};

// The rope part of a lane, 16 values of key lane / 4, into the 64 keys x 64 dimensions at `block`.
__device__ __forceinline__ void store_rope(const uint4& rope, uint32_t block, int w, int lane) {
  const uint32_t words[4] = {rope.x, rope.y, rope.z, rope.w};
  uint32_t h[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    h[2 * q] = e4m3x2_to_f16x2(static_cast<uint16_t>(words[q] & 0xFFFFu));
    h[2 * q + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(words[q] >> 16));
  }
  const uint32_t key = 8u * w + (lane >> 2), col = 2 * (lane & 3);
  st_shared_v4(block + swizzled(key, col), h[0], h[1], h[2], h[3]);
  st_shared_v4(block + swizzled(key, col + 1), h[4], h[5], h[6], h[7]);
}

// Q of a score CTA's 128 rows (from row r0 of all, `rows` of them exist), as FP16: the
// latent part into tensor memory, the rope part into shared memory. Two of the
// eight warps share a quarter of the rows: half of the blocks each. Four lanes load
// 64 bytes of a row at a time.
struct QLoad {
  const uint16_t* lat;   // the lane's first row and dimensions
  const uint16_t* rope;
  int32_t left;          // rows from the lane's first one on
  uint32_t v[2][8];      // of two rows, 8 apart

  __device__ __forceinline__ QLoad(const ChunkParams& p, int64_t row0, int32_t rows, int first, int lane) {
    const int r = first + (lane >> 2);
    lat = p.q_lat + (row0 + r) * kLatent + 8 * (lane & 3);
    rope = p.q_rope + (row0 + r) * kRope + 8 * (lane & 3);
    left = rows - r;
  }
  // rows 16 y + {0, 8} of 64 dimensions
  __device__ __forceinline__ void load(const uint16_t* from, int width, int y) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[z][k] = 0u;
      if (left > 16 * y + 8 * z) ld_two_v4(from + (16 * y + 8 * z) * width, v[z]);
    }
  }
};

// Partial results lie in the order in which a warp has them (as rows of 512 values they took
// 8.4 us to write, 128 rows a CTA, and 4.4 in this order): of 8 rows and 64
// dimensions four times 32 lanes' 16 bytes; lane 4 (row % 8) + c of number q has
// dimensions 32 (q / 2) + 8 c + 4 (q % 2) .. + 3. Here the place of 8 rows' first.
__device__ __forceinline__ int64_t part_at(int32_t slot, int row) {
  return (static_cast<int64_t>(slot) * kTileRows + row) * (kLatent / 4);
}

// ------------------------------------------------------------------ kernel
template <int kFmt>
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kChunkThreads, 1) chunk_kernel(const ChunkParams p) {
  using L = ChunkLayout<kFmt>;
  using C = ChunkCtl;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ctl = sbase + L::kCtl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = static_cast<int>(blockIdx.x) / 4;
  const bool scoring = rank < 2;
  const uint32_t part = rank & 1;  // which of the pair; the leader is 0
  const long long lim = p.wait_cycles;
  const uint32_t abort_addr = ctl + C::kAbort;
  auto bar = [&](uint32_t off, uint32_t i) { return ctl + off + 8u * i; };

  if (tid == 0) {
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(bar(C::kRawFull, i), 1);
      mbar_init(bar(C::kRawEmpty, i), kExpandWarps);
      mbar_init(bar(C::kKFull, i), kExpandWarps);
      mbar_init(bar(C::kPeer, i), 1);
      mbar_init(bar(C::kSFull, i), 1);
      mbar_init(bar(C::kSEmpty, i), 8);  // four warps a piece
      mbar_init(bar(C::kKHalf, i), 1);
    }
    mbar_init(bar(C::kQFull, 0), kExpandWarps);
    for (uint32_t i = 0; i < 4 * kGroups; ++i) mbar_init(bar(C::kRefDone, i), 1);
    for (uint32_t i = 0; i < 16 * kGroups; ++i) mbar_init(bar(C::kSumDone, i), 1);
    for (uint32_t i = 0; i < L::kStages; ++i) mbar_init(bar(C::kStaged, i), 4);
    for (uint32_t i = 0; i < 4; ++i) mbar_init(bar(C::kStageFree, i), 1);
    for (uint32_t i = 0; i < L::kPSlots; ++i) {
      mbar_init(bar(C::kPFull, i), 1);
      mbar_init(bar(C::kPReady, i), 1);
      mbar_init(bar(C::kPvDone, i), 1);
    }
    for (uint32_t i = 0; i < L::kVSlots; ++i) mbar_init(bar(C::kVFull, i), kExpandWarps);
    mbar_init(bar(C::kTask, 0), 1);
    mbar_init(bar(C::kTaskDone, 0), kSoftWarps);
    st_shared_u32(ctl + C::kSent, 0u);
    st_shared_u32(ctl + C::kScored, 0u);
    st_shared_u32(ctl + C::kSummed, 0u);
    st_shared_u32(ctl + C::kLoaded, 0u);
    for (uint32_t i = 0; i < 4; ++i) st_shared_u32(ctl + C::kNoted + 4 * i, 0u);
    st_shared_u32(abort_addr, (sbase & 1023u) != 0 ? 1u : 0u);
    fence_mbar_init();
  }
  if (tid < 8 * C::kMissingTiles) st_shared_u32(ctl + C::kMissing + 4 * tid, 0u);
  if (!scoring && tid < 4 * L::kNotes) st_shared_u32(sbase + L::kTag + 4 * tid, 0u);
  if (warp == kIssueWarp) alloc_tmem_pair(ctl + C::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the other CTAs' barriers exist before anyone arrives on them
  const uint32_t tmem = ld_shared_u32(ctl + C::kTmem);
  if (tmem != 0u && tid == 0) st_shared_u32(abort_addr, 1u);  // the operands assume base 0
  cudaGridDependencySynchronize();  // the plan is there
  cudaTriggerProgrammaticLaunchCompletion();

  // All warps of a warpgroup change their registers together.
  if (warp >= kIssueWarp) {
    set_registers<kIssueRegs>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------- cache rows, 64 keys at a time
      // A score CTA loads its 64 keys of each tile, an output CTA all keys. Pages of
      // a multiple of 64 rows hold them in one run, copied whole: what lies behind
      // the length is seen by no row. Other pages go row by row.
      const uint32_t raws = scoring ? L::kRawsScore : L::kRawsOut;
      const uint32_t raw = sbase + (scoring ? L::kRawScore : L::kRawOut);
      const bool runs = p.page.size % kPieceKeys == 0;
      uint32_t u = 0;
      bool run = true;
      Pieces pieces(p, cluster);
      while (run && pieces.next()) {
        // the next row tile's Q, into L2
        if (scoring && lane < 2 && pieces.t < pieces.tiles && p.tiles[pieces.t].unit < pieces.u1) {
          const RowTile& after = p.tiles[pieces.t];
          const int32_t rows = min(after.rows - 128 * static_cast<int32_t>(part), 128);
          const int64_t first = after.row0 + 128 * part;
          if (rows > 0)
            prefetch_l2(lane == 0 ? p.q_lat + first * kLatent : p.q_rope + first * kRope,
                        static_cast<uint32_t>(rows) * 2u * (lane == 0 ? kLatent : kRope));
        }
        __syncwarp();
        const int32_t* table = p.block_table + static_cast<int64_t>(pieces.tile.seq) * p.max_blocks;
        const int32_t step = scoring ? kTileKeys : kPieceKeys;
        const int32_t stop = pieces.end * kTileKeys;
        int32_t key = pieces.begin * kTileKeys + (scoring ? kPieceKeys * static_cast<int32_t>(part) : 0);
        auto page_of = [&](int32_t k) { return k < pieces.tile.len && k < stop ? __ldg(table + p.page.block(k)) : -1; };
        int32_t page = runs ? page_of(key) : 0;
        for (; key < stop; key += step, ++u) {
          const uint32_t s = u % raws;
          const int32_t next = runs ? page_of(key + step) : 0;
          if (u >= raws && !warp_wait(bar(C::kRawEmpty, s), ((u / raws) & 1) ^ 1, abort_addr, lim)) {
            run = false;
            break;
          }
          const uint32_t dst = raw + s * L::kRawBytes, full = bar(C::kRawFull, s);
          // bits of the keys that exist, and of those among them without a page
          uint32_t have[2], lost[2];
          int64_t off[2];
          if (runs) {
            const bool ok = page >= 0 && page < p.num_blocks;
            const int32_t left = pieces.tile.len - key;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              have[x] = ok ? 0xffffffffu : 0u;
              lost[x] = !ok && left > 32 * x ? 0xffffffffu : 0u;
            }
            off[0] = page * p.block_stride +
                     static_cast<int64_t>(key - p.page.block(key) * p.page.size) * static_cast<int64_t>(L::kRow);
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int32_t k = key + 32 * x + lane;
              const bool some = k < pieces.tile.len;
              const int32_t b = some ? p.page.block(k) : 0;
              const int32_t id = some ? __ldg(table + b) : -1;
              const bool ok = id >= 0 && id < p.num_blocks;
              off[x] = id * p.block_stride +
                       static_cast<int64_t>(k - b * p.page.size) * static_cast<int64_t>(L::kRow);
              have[x] = __ballot_sync(0xffffffffu, ok);
              lost[x] = __ballot_sync(0xffffffffu, some && !ok);
            }
          }
          if (scoring && (lost[0] | lost[1]) != 0u) {  // the softmax of both CTAs has to know
            if (lane < 2) {
              const uint32_t to = map_rank(ctl + C::kMissing + 32 * (u % C::kMissingTiles) + 16 * part, lane);
              st_cluster_u32(to + 4, ~lost[0]);
              st_cluster_u32(to + 8, ~lost[1]);
            }
            fence_cluster();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_tx(full, static_cast<uint32_t>(__popc(have[0]) + __popc(have[1])) * L::kRow);
          __syncwarp();
          if (runs) {
            if (lane == 0 && have[0] != 0u) bulk_g2s(dst, p.cache + off[0], L::kRawBytes, full);
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if ((have[x] >> lane) & 1u) bulk_g2s(dst + (32 * x + lane) * L::kRow, p.cache + off[x], L::kRow, full);
          }
          // Behind the copies: the next arrival waits until the word has landed. In front of them
          // 66 single tokens with FP8 rows took 641 us, in place of 561.
          if (scoring && lane < 2)
            st_relaxed_cluster(map_rank(ctl + C::kMissing + 32 * (u % C::kMissingTiles) + 16 * part, lane),
                               2 * (u + 1) + ((lost[0] | lost[1]) != 0u ? 1u : 0u));
          __syncwarp();
          page = next;
        }
      }
      if (lane == 0) st_shared_u32(ctl + C::kLoaded, u);
    } else if (warp == kSendWarp && scoring) {
      // ---------------------------------------------- P pieces to the output CTA
      const uint32_t out_p = map_rank(sbase + L::kP, 2 + part), out_full = map_rank(bar(C::kPFull, 0), 2 + part);
      uint32_t u = 0;
      bool run = true;
      Pieces pieces(p, cluster);
      while (run && pieces.next()) {
        const uint32_t n = static_cast<uint32_t>(pieces.end - pieces.begin) * 2;
        for (uint32_t x = 0; x < n; ++x, ++u) {
          const uint32_t ps = u % L::kPSlots, st = u % L::kStages;
          run = warp_wait(bar(C::kStaged, st), (u / L::kStages) & 1, abort_addr, lim) &&
                (u < L::kPSlots ||
                 warp_wait<true>(bar(C::kPvDone, ps), ((u / L::kPSlots) & 1) ^ 1, abort_addr, lim));
          if (!run) break;
          const bool noted = ld_shared_u32(ctl + C::kNoted + 4 * (u & 3)) == u + 1;
          if (noted) fence_cluster();  // the notes are there first
          if (elect_one())
            bulk_s2s(out_p + ps * kPBytes, sbase + L::kStaged + st * kPBytes, kPBytes, out_full + 8u * ps);
          __syncwarp();
        }
      }
      if (lane == 0) st_cluster_u32(map_rank(ctl + C::kSent, 2 + part), u);
    } else if (warp == kSendWarp) {
      // ---------------------------------------------- P pieces have left their stage
      // and their slots' barriers take the next one, in this CTA: an arrival from the
      // score CTA would cost its sender 300 cycles a piece.
      if (lane == 0)
        for (uint32_t i = 0; i < L::kPSlots; ++i) mbar_arrive_tx(bar(C::kPFull, i), kPBytes);
      const uint32_t freed = map_rank(bar(C::kStageFree, 0), part);
      uint32_t u = 0;
      bool run = true;
      Pieces pieces(p, cluster);
      while (run && pieces.next()) {
        const uint32_t n = static_cast<uint32_t>(pieces.end - pieces.begin) * 2;
        for (uint32_t x = 0; x < n; ++x, ++u) {
          run = warp_wait<true>(bar(C::kPFull, u % L::kPSlots), (u / L::kPSlots) & 1, abort_addr, lim);
          if (!run) break;
          if (elect_one()) {
            mbar_arrive_cluster_relaxed(freed + 8u * (u & 3));
            mbar_arrive_tx(bar(C::kPFull, u % L::kPSlots), kPBytes);
          }
          __syncwarp();
        }
      }
    } else if (warp == kIssueWarp && scoring) {
      // ---------------------------------------------- S = Q K^T
      // The leader's warp issues the MMAs, the other one tells it what its CTA has
      // ready. The whole warp goes through the loop, so that operands stay uniform.
      constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(kTileKeys >> 3) << 17) |
                                  (static_cast<uint32_t>(kTileRows >> 4) << 24);
      const uint64_t qr = operand_desc(sbase + L::kQRope);
      const uint32_t peer = map_rank(bar(C::kPeer, 0), 0);
      const uint64_t k0 = operand_desc(sbase + L::kK);
      uint32_t i = 0, first = 0;  // ring position of the tile's first block
      bool run = true;
      Pieces pieces(p, cluster);
      for (uint32_t item = 0; run && pieces.next(); ++item) {
        if (!warp_wait(bar(C::kQFull, 0), item & 1, abort_addr, lim)) break;
        for (int32_t kt = pieces.begin; kt < pieces.end; ++kt, ++i) {
          const uint32_t b = i & 1, ph = (i >> 1) & 1;
          run = warp_wait(bar(C::kSEmpty, b), ph ^ 1, abort_addr, lim) &&
                warp_wait(bar(C::kKFull, b), ph, abort_addr, lim);
          if (!run) break;
          tc_fence_after();
          if (part != 0) {
            tc_fence_before();
            if (elect_one()) arrive_remote(peer + 8u * b);
            __syncwarp();
            continue;
          }
          run = warp_wait<true>(bar(C::kPeer, b), ph, abort_addr, lim);
          if (!run) break;
          tc_fence_after();
          const uint32_t d = kSCol + kTileKeys * b;
          if (elect_one()) {
            uint32_t at = first;
#pragma unroll
            for (uint32_t block = 0; block < kTileBlocks; ++block) {
              const uint64_t kd = k0 + at * (kKBlock >> 4);
#pragma unroll
              for (uint32_t x = 0; x < 4; ++x) {
                if (block < 8) pair_mma_ts(d, 32 * block + 8 * x, kd + 2 * x, kIdesc, (block | x) != 0 ? 1u : 0u);
                else pair_mma_ss(d, qr + 2 * x, kd + 2 * x, kIdesc, 1u);
              }
              if (block + 1 == L::kKShared) commit_to(bar(C::kKHalf, b), 0x3);
              if (++at == L::kKBlocks) at = 0;
            }
            commit_to(bar(C::kSFull, b), 0x3);
          }
          __syncwarp();
          first = (first + kTileBlocks) % L::kKBlocks;
        }
      }
      if (part == 0 && lane < 2) st_cluster_u32(map_rank(ctl + C::kScored, lane), i);
    } else if (warp == kIssueWarp) {
      // ---------------------------------------------- O += P V
      // The warp follows the P pieces that land in its CTA, has O rescaled where a
      // piece comes with factors and written behind the last piece of a row tile
      // (tasks of the twelve rescaling warps); then the leader's issues the MMAs and
      // the other one tells it.
      constexpr uint32_t kIdesc = (1u << 4) | (1u << 16) | ((256u >> 3) << 17) |
                                  (static_cast<uint32_t>(kTileRows >> 4) << 24);
      const uint32_t peer = map_rank(bar(C::kPReady, 0), 2);
      uint32_t u = 0, tasks = 0;
      bool run = true;
      auto post = [&](uint32_t word) {
        if (lane == 0) {
          st_shared_u32(ctl + C::kTaskWord, word);
          mbar_arrive(bar(C::kTask, 0));
        }
        __syncwarp();
        ++tasks;
      };
      auto task_done = [&]() { return warp_wait(bar(C::kTaskDone, 0), (tasks - 1) & 1, abort_addr, lim); };
      Pieces pieces(p, cluster);
      while (run && pieces.next()) {
        const uint32_t n = static_cast<uint32_t>(pieces.end - pieces.begin) * 2;
        if (tasks > 0 && !task_done()) break;  // O before has been read
        for (uint32_t x = 0; x < n; ++x, ++u) {
          const uint32_t ps = u % L::kPSlots, vs = u % L::kVSlots;
          run = warp_wait<true>(bar(C::kPFull, ps), (u / L::kPSlots) & 1, abort_addr, lim);
          if (!run) break;
          const uint4 tag = ld_shared_v4(sbase + L::kTag + 16 * (u % L::kNotes));
          if (tag.x == u + 1 || tag.y == u + 1 || tag.z == u + 1 || tag.w == u + 1) {
            post(2 * u);
            run = task_done();
            if (!run) break;
          }
          run = warp_wait(bar(C::kVFull, vs), (u / L::kVSlots) & 1, abort_addr, lim);
          if (!run) break;
          tc_fence_after();
          if (part != 0) {
            tc_fence_before();
            if (elect_one()) arrive_remote(peer + 8u * ps);
            __syncwarp();
            continue;
          }
          run = warp_wait<true>(bar(C::kPReady, ps), (u / L::kPSlots) & 1, abort_addr, lim);
          if (!run) break;
          tc_fence_after();
          const uint64_t pd = operand_desc(sbase + L::kP + ps * kPBytes);
          const uint64_t vd = operand_desc(sbase + L::kV + vs * kVSlotBytes, kKBlock);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int nh = 0; nh < 2; ++nh)
                pair_mma_ss(256u * nh, pd + 2 * kk, vd + nh * (kVSlotBytes >> 5) + kk * (2048 >> 4), kIdesc,
                            (x | kk) != 0 ? 1u : 0u);
            commit_to(bar(C::kPvDone, ps), 0xF);
          }
          __syncwarp();
        }
        if (run) post(2 * (u - 1) + 1);
      }
      if (part == 0 && lane < 4) st_cluster_u32(map_rank(ctl + C::kSummed, lane), u);
    }
  } else if (warp >= kExpandWarp0) {
    set_registers<kExpandRegs>();
    const int w = warp - kExpandWarp0;
    uint32_t u = 0;
    bool run = true;
    Pieces pieces(p, cluster);
    if (scoring) {
      // ---------------------------------------------- keys of a score CTA
      // Tile u goes into the ring once the MMAs of tile u - 2 are done, its last blocks
      // once those of tile u - 1's first kKShared are.
      uint32_t first = 0;  // ring position of the tile's first block
      while (run && pieces.next()) {
        for (int32_t kt = pieces.begin; kt < pieces.end; ++kt, ++u) {
          const uint32_t s = u % L::kRawsScore;
          run = warp_wait(bar(C::kRawFull, s), (u / L::kRawsScore) & 1, abort_addr, lim);
          if (!run) break;
          RowItems<kFmt, true> items;
          items.load(sbase + L::kRawScore + s * L::kRawBytes, w, lane, 0);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kRawEmpty, s));
          run = u < 2 || warp_wait(bar(C::kSFull, u & 1), ((u >> 1) & 1) ^ 1, abort_addr, lim);
          if (!run) break;
          auto block_at = [&](uint32_t block) {
            const uint32_t at = first + block;
            return sbase + L::kK + (at < L::kKBlocks ? at : at - L::kKBlocks) * kKBlock;
          };
          items.store_blocks(0, block_at, w, lane);
          if (u > 0) {
            run = warp_wait(bar(C::kKHalf, (u - 1) & 1), ((u - 1) >> 1) & 1, abort_addr, lim);
            if (!run) break;
          }
          items.store_blocks(1, block_at, w, lane);
          store_rope(items.rope, block_at(8), w, lane);
          first = (first + kTileBlocks) % L::kKBlocks;
          fence_proxy_async_cta();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kKFull, u & 1));
          if (kt == pieces.begin) {  // Q, once the MMAs of the row tile before are done with its
            const uint32_t quad = w & 3, half = w >> 2;
            QLoad a(p, pieces.tile.row0, pieces.tile.rows, 128 * part + 32 * quad, lane), b = a;
            const uint32_t q_addr = tmem + ((32 * quad) << 16) + 128 * half;
            auto put = [&](const QLoad& q, int x) {  // rows 16 (x % 2) .. + 15 of block 4 half + x / 2
              uint32_t h[16];
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  h[4 * j + z] = to_f16x2(q.v[0][2 * j + z], p.lat_mult);
                  h[4 * j + 2 + z] = to_f16x2(q.v[1][2 * j + z], p.lat_mult);
                }
              tmem_st_16x256b_x4(q_addr + ((16 * (x & 1)) << 16) + 32u * (x >> 1), h);
            };
            a.load(a.lat + 256 * half, kLatent, 0);
            b.load(b.lat + 256 * half, kLatent, 1);
            if (u > 0) run = warp_wait(bar(C::kSFull, (u - 1) & 1), ((u - 1) >> 1) & 1, abort_addr, lim);
            if (!run) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < 8; x += 2) {
              put(a, x);
              if (x < 6) a.load(a.lat + 256 * half + 32 * (x + 2), kLatent, 0);
              else a.load(a.rope, kRope, half);
              put(b, x + 1);
              if (x < 6) b.load(b.lat + 256 * half + 32 * (x + 2), kLatent, 1);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t r = 32 * quad + 16 * half + 8 * z + (lane >> 2), col = lane & 3;
              uint32_t h[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) h[k] = to_f16x2(a.v[z][k], p.rope_mult);
              st_shared_v4(sbase + L::kQRope + swizzled(r, col), h[0], h[1], h[2], h[3]);
              st_shared_v4(sbase + L::kQRope + swizzled(r, col + 4), h[4], h[5], h[6], h[7]);
            }
            tmem_st_wait();
            tc_fence_before();
            fence_proxy_async_cta();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kQFull, 0));
          }
        }
      }
    } else {
      // ---------------------------------------------- values of an output CTA
      // Piece u goes into slot u % kVSlots, once the MMAs of piece u - kVSlots are done.
      while (run && pieces.next()) {
        const int32_t stop = 2 * pieces.end;
        for (int32_t x = 2 * pieces.begin; x < stop; ++x, ++u) {
          const uint32_t s = u % L::kRawsOut, vs = u % L::kVSlots;
          run = warp_wait(bar(C::kRawFull, s), (u / L::kRawsOut) & 1, abort_addr, lim);
          if (!run) break;
          RowItems<kFmt, false> items;
          items.load(sbase + L::kRawOut + s * L::kRawBytes, w, lane, part);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kRawEmpty, s));
          const uint32_t v = u - L::kVSlots;
          run = u < L::kVSlots ||
                warp_wait<true>(bar(C::kPvDone, v % L::kPSlots), (v / L::kPSlots) & 1, abort_addr, lim);
          if (!run) break;
          items.store_blocks(0, [&](uint32_t block) { return sbase + L::kV + vs * kVSlotBytes + block * kKBlock; },
                             w, lane);
          fence_proxy_async_cta();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kVFull, vs));
        }
      }
    }
  } else {
    set_registers<kSoftRegs>();
    const uint32_t group = warp >> 2, quad = warp & 3;
    const uint32_t t = tid & 127;
    const uint32_t lane_base = (32 * quad) << 16;
    const int row = 128 * static_cast<int>(part) + static_cast<int>(t);  // of the row tile
    bool ok = true;
    Pieces pieces(p, cluster);
    if (scoring) {
      // ---------------------------------------------- softmax (thread = row)
      // The groups of four warps take the pieces in turn: one has the time of three
      // pieces for each. A row's reference goes from piece to piece through shared
      // memory; each group has a sum of its own.
      const uint32_t out_rank = 2 + part;
      const float c = p.score_scale;
      const uint64_t c2 = f32x2(c, c);
      uint32_t i0 = 0;  // tiles before
      for (uint32_t item = 0; ok && pieces.next(); ++item) {
        const uint32_t n = static_cast<uint32_t>(pieces.end - pieces.begin) * 2;
        // keys that the row sees
        const int32_t sees =
            pieces.tile.base + 1 + (pieces.tile.offset + min(row, pieces.tile.rows - 1)) / p.num_heads;
        float m = -INFINITY, l = 0.f;  // the reference that l is relative to
        for (uint32_t x = (group + kGroups - 2 * i0 % kGroups) % kGroups; x < n; x += kGroups) {
          const uint32_t u = 2 * i0 + x, i = u >> 1, b = i & 1, half = u & 1, st = u % L::kStages;
          ok = warp_wait(bar(C::kSFull, b), (i >> 1) & 1, abort_addr, lim);
          if (!ok) break;
          tc_fence_after();
          uint32_t s[2][32];
          const uint32_t s_addr = tmem + lane_base + kSCol + kTileKeys * b + kPieceKeys * half;
          tmem_ld32(s_addr, s[0]);
          tmem_ld32(s_addr + 32u, s[1]);
          // keys of the piece that the row could see, and those that exist
          const int32_t room = sees - pieces.begin * kTileKeys - kPieceKeys * static_cast<int32_t>(x);
          const uint32_t word_at = ctl + C::kMissing + 32 * (i % C::kMissingTiles) + 16 * half;
          uint32_t word = ld_relaxed_cluster(word_at);
          tmem_ld_wait();
          // one branch for the warp: a test at each score cost more than the exponentials
          const bool all = __all_sync(0xffffffffu, room >= kPieceKeys && word == 2 * (i + 1));
          uint32_t bits[2] = {0xffffffffu, 0xffffffffu};
          if (!all) {
            ok = warp_wait_word(word_at, i, word, abort_addr, lim);
            if (!ok) break;
            if (word & 1u) {
              fence_cluster();
              bits[0] = ld_shared_u32(word_at + 4);
              bits[1] = ld_shared_u32(word_at + 8);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kSEmpty, b));  // S is read
          if (!all) {  // the keys that the row sees
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              const int32_t seen = room - 32 * a;
              if (seen < 32) bits[a] = seen <= 0 ? 0u : bits[a] & ((1u << seen) - 1u);
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (!((bits[a] >> y) & 1u)) s[a][y] = 0xff800000u;  // -inf
            }
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int y = 0; y < 32; y += 4) {
            tops[0] = fmax3(tops[0], __uint_as_float(s[0][y]), __uint_as_float(s[0][y + 1]));
            tops[1] = fmax3(tops[1], __uint_as_float(s[0][y + 2]), __uint_as_float(s[0][y + 3]));
            tops[2] = fmax3(tops[2], __uint_as_float(s[1][y]), __uint_as_float(s[1][y + 1]));
            tops[3] = fmax3(tops[3], __uint_as_float(s[1][y + 2]), __uint_as_float(s[1][y + 3]));
          }
          const float mx = fmaxf(fmax3(tops[0], tops[1], tops[2]), tops[3]);
          const float top = mx == -INFINITY ? -INFINITY : mx * c;
          // the reference behind the piece before, and behind this one
          if (u > 0) {
            const uint32_t v = u - 1;
            ok = warp_wait(bar(C::kRefDone, 4 * (v % kGroups) + quad), (v / kGroups) & 1, abort_addr, lim);
            if (!ok) break;
          }
          const uint32_t ref_at = sbase + L::kRef + 4 * t;
          auto ref_of = [&](uint32_t v) { return __uint_as_float(ld_shared_u32(ref_at + 512 * (v % kGroups))); };
          const float before = x > 0 ? ref_of(u - 1) : -INFINITY;
          const bool last = x + 1 == n;
          const float earlier = last && x > 1 ? ref_of(u - 2) : -INFINITY;  // while it is there
          const bool moves = top > before + kTau;  // also the first score that the row sees
          const float ref = moves ? top - kHeadroom : before;
          st_shared_u32(ref_at + 512 * group, __float_as_uint(ref));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kRefDone, 4 * group + quad));
          if (ref != m) {
            l *= m == -INFINITY ? 0.f : ex2(m - ref);
            m = ref;
          }
          const float nm = m == -INFINITY ? 0.f : -m;
          const uint64_t nm2 = f32x2(nm, nm);
          uint32_t pk[2][16];
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              float e0, e1;
              split_f32x2(
                  fma_f32x2(f32x2(__uint_as_float(s[a][2 * y]), __uint_as_float(s[a][2 * y + 1])), c2, nm2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum[y & 1] = add_f32x2(sum[y & 1], f32x2(e0, e1));
              pk[a][y] = pack_f16x2(e0, e1);
            }
          {
            float e0, e1;
            split_f32x2(add_f32x2(sum[0], sum[1]), e0, e1);
            l += e0 + e1;
          }
          if (u >= L::kStages) {  // the stage's piece before has left it
            const uint32_t v = u - L::kStages;
            ok = warp_wait<true>(bar(C::kStageFree, v & 3), (v >> 2) & 1, abort_addr, lim);
            if (!ok) break;
          }
          const uint32_t dst = sbase + L::kStaged + st * kPBytes;
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              st_shared_v4(dst + swizzled(t, 4 * a + q), pk[a][4 * q], pk[a][4 * q + 1], pk[a][4 * q + 2],
                           pk[a][4 * q + 3]);
          // What goes with the piece, rarely: factors, and behind the last one what the
          // output is to be multiplied by
          const bool rescale = __any_sync(0xffffffffu, moves && before != -INFINITY);
          if (rescale || last) {
            if (rescale) {
              const uint32_t note = u % L::kNotes;
              const float alpha = !moves ? 1.f : before == -INFINITY ? 0.f : ex2(before - ref);
              st_cluster_u32(map_rank(sbase + L::kFactor + 512 * note + 4 * t, out_rank), __float_as_uint(alpha));
              if (lane == 0) st_cluster_u32(map_rank(sbase + L::kTag + 16 * note + 4 * quad, out_rank), u + 1);
            }
            if (last) {
              for (uint32_t d = 1; d < kGroups && ok; ++d) {  // the group of piece u - d
                const uint32_t g = (group + kGroups - d) % kGroups;
                ok = warp_wait(bar(C::kSumDone, 4 * kGroups * (item & 3) + 4 * g + quad), (item >> 2) & 1,
                               abort_addr, lim);
                const float other =
                    __uint_as_float(ld_shared_u32(sbase + L::kSums + 512 * (kGroups * (item & 3) + g) + 4 * t));
                if (other != 0.f) l += other * ex2((d == 1 ? before : earlier) - ref);
              }
              if (!ok) break;
              st_cluster_u32(map_rank(sbase + L::kFinal + 512 * (item % L::kNotes) + 4 * t, out_rank),
                             __float_as_uint(l == 0.f ? 0.f : p.out_mult / l));
            }
            if (lane == 0) st_shared_u32(ctl + C::kNoted + 4 * (u & 3), u + 1);
          }
          fence_proxy_async_cta();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kStaged, st));
          if (last && row < pieces.tile.rows) {
            const float lse = l == 0.f ? -INFINITY : (m + lg2(l)) * kLn2;
            if (!pieces.whole) p.part_lse[static_cast<int64_t>(pieces.slot) * kTileRows + row] = lse;
            else if (p.lse != nullptr) p.lse[pieces.tile.row0 + row] = lse;
          }
        }
        if (!ok) break;
        // for the group that ends the result (nobody waits for that one's own)
        st_shared_u32(sbase + L::kSums + 512 * (kGroups * (item & 3) + group) + 4 * t, __float_as_uint(l));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kSumDone, 4 * kGroups * (item & 3) + 4 * group + quad));
        i0 += n / 2;
      }
    } else {
      // ---------------------------------------------- rescaling and output (thread = row)
      // The groups of four warps take blocks of 32 columns in turn.
      const uint32_t o_addr = tmem + lane_base;
      uint32_t tasks = 0;
      for (uint32_t item = 0; ok && pieces.next(); ++item) {
        // A result may come with its last piece only: the wait for it is as long as those of
        // all pieces, each of which other warps wait for.
        const long long n = 2ll * (pieces.end - pieces.begin);
        const long long all = lim < (1ll << 62) / n ? lim * n : 1ll << 62;
        for (bool rescaling = true; rescaling;) {
          ok = warp_wait(bar(C::kTask, 0), tasks & 1, abort_addr, all);
          if (!ok) break;
          ++tasks;
          const uint32_t word = ld_shared_u32(ctl + C::kTaskWord);
          const uint32_t u = word >> 1, ps = u % L::kPSlots, note = u % L::kNotes;
          rescaling = (word & 1u) == 0u;
          if (rescaling) {
            if (ld_shared_u32(sbase + L::kTag + 16 * note + 4 * quad) == u + 1) {
              // behind a piece of the same rows, whose MMAs (and all before) have to be done
              const uint32_t v = u - 1;
              ok = warp_wait<true>(bar(C::kPvDone, v % L::kPSlots), (v / L::kPSlots) & 1, abort_addr, lim);
              if (!ok) break;
              tc_fence_after();
              const float alpha = __uint_as_float(ld_shared_u32(sbase + L::kFactor + 512 * note + 4 * t));
#pragma unroll 1
              for (uint32_t y = group; y < 16; y += kGroups) {
                uint32_t r[32];
                tmem_ld32(o_addr + 32u * y, r);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 32; ++q) r[q] = __float_as_uint(__uint_as_float(r[q]) * alpha);
                tmem_st32(o_addr + 32u * y, r);
              }
              tmem_st_wait();
            }
          } else {
            ok = warp_wait<true>(bar(C::kPvDone, ps), (u / L::kPSlots) & 1, abort_addr, lim);
            if (!ok) break;
            tc_fence_after();
            // 16 rows x 64 dimensions at a time: a lane has twice 8 dimensions of two rows
            const uint32_t finals = sbase + L::kFinal + 512 * (item % L::kNotes) + 4 * (32 * quad + (lane >> 2));
            const int r0 = 128 * static_cast<int>(part) + 32 * static_cast<int>(quad) + (lane >> 2);
            float* wide = static_cast<float*>(p.out) + (pieces.tile.row0 + r0) * kLatent + 8 * (lane & 3);
            float4* parts = reinterpret_cast<float4*>(p.part_out) +
                            part_at(pieces.slot, 128 * static_cast<int>(part) + 32 * static_cast<int>(quad)) + lane;
            uint16_t* narrow = static_cast<uint16_t*>(p.out) + (pieces.tile.row0 + r0) * kLatent + 8 * (lane & 3);
#pragma unroll 1
            for (uint32_t y = group; y < 16; y += kGroups) {
              const uint32_t block = y >> 1, rows = 16 * (y & 1);
              uint32_t r[32];
              tmem_ld_16x256b_x8(o_addr + (rows << 16) + 64u * block, r);
              tmem_ld_wait();
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int at = static_cast<int>(rows) + 8 * z;
                const float fin = __uint_as_float(ld_shared_u32(finals + 4 * at));
                float v[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  v[2 * j] = __uint_as_float(r[4 * j + 2 * z]) * fin;
                  v[2 * j + 1] = __uint_as_float(r[4 * j + 2 * z + 1]) * fin;
                }
                if (r0 + at >= pieces.tile.rows) continue;
                const int64_t to = static_cast<int64_t>(at) * kLatent + 64 * block;
                if (!pieces.whole) {
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    parts[128 * (8 * (at >> 3) + block) + 32 * q] =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                } else if (p.out_fp32) {
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<float4*>(wide + to + 32 * (q >> 1) + 4 * (q & 1)) =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                } else {
#pragma unroll
                  for (int q = 0; q < 2; ++q)
                    *reinterpret_cast<uint4*>(narrow + to + 32 * q) =
                        make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                   pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kTaskDone, 0));
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  // Every CTA now knows what was issued towards it, also by a cluster that gave
  // up; it waits (bounded) until that has landed, before its memory goes away.
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && ld_shared_u32(abort_addr) != 0u) p.failed[cluster] = 1;
  cluster_sync();
  if (tid == 0) {
    auto drain_last = [&](uint32_t off, uint32_t count, uint32_t slots) {
      if (count > 0) drain(bar(off, (count - 1) % slots), ((count - 1) / slots) & 1);
    };
    drain_last(C::kSFull, ld_shared_u32(ctl + C::kScored), 2);
    drain_last(C::kPFull, ld_shared_u32(ctl + C::kSent), L::kPSlots);
    drain_last(C::kPvDone, ld_shared_u32(ctl + C::kSummed), L::kPSlots);
    const uint32_t loaded = ld_shared_u32(ctl + C::kLoaded), raws = scoring ? L::kRawsScore : L::kRawsOut;
    for (uint32_t s = 0; s < raws && s < loaded; ++s) drain_last(C::kRawFull, loaded - s, raws);
  }
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    free_tmem_pair(tmem);
  }
  cluster_sync();
}

// ------------------------------------------------------------------ merging
// Row tiles that several clusters worked on: out = sum_p w_p out_p / sum_p w_p
// with w_p = exp(lse_p - max). A warp has a row; the border between two
// clusters' shares that is the first inside a row tile stands for it.
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p) {
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  const int64_t me = static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x;  // few rows: an SM each
  bool failed = false;
  for (int c = lane; c < p.clusters; c += 32) failed |= __ldcg(p.failed + c) != 0;
  if (__any_sync(0xffffffffu, failed)) {  // a wait ran out: no row is to be trusted
    for (int s = 0; s < p.num_seqs; ++s) {
      int32_t start, len;
      const int64_t n = static_cast<int64_t>(new_tokens(p, s, start, len)) * p.num_heads;
      for (int64_t r = me; r < n; r += warps) {
        const int64_t at = static_cast<int64_t>(start) * p.num_heads + r;
        for (int d = lane; d < kLatent; d += 32) {
          if (p.out_fp32) static_cast<float*>(p.out)[at * kLatent + d] = NAN;
          else static_cast<uint16_t*>(p.out)[at * kLatent + d] = 0x7FFF;
        }
        if (lane == 0 && p.lse != nullptr) p.lse[at] = NAN;
      }
    }
    return;
  }
  const int64_t units = __ldcg(&p.plan->units), share = __ldcg(&p.plan->share);
  for (int64_t x = me; x < static_cast<int64_t>(p.clusters - 1) * kTileRows; x += warps) {
    const int c = 1 + static_cast<int>(x / kTileRows), row = static_cast<int>(x % kTileRows);
    const int64_t at = c * share;
    if (at >= units) break;
    const int t = __ldcg(p.first + c);  // whose units reach to c's first one, or begin there
    // first[c] is the last row tile that begins at or before `at`
    const RowTile tile = p.tiles[t];
    const int64_t a = tile.unit, b = tile.end;
    if (a == at || a < at - share || row >= tile.rows) continue;  // not cut here, or before
    const int64_t k0 = a + kTileOverhead;
    const int c1 = static_cast<int>((b - 1) / share);
    // the parts: cluster c - 1 to c1, those that have key tiles
    auto has = [&](int q) {
      const int64_t lo = max(q * share - k0, int64_t{0}), hi = min((q + 1) * share, b) - k0;
      return hi > lo;
    };
    auto lse_at = [&](int q) {
      return p.part_lse + static_cast<int64_t>(2 * q + (a >= q * share ? 1 : 0)) * kTileRows + row;
    };
    int q0 = c - 1;
    while (q0 < c1 && !has(q0)) ++q0;
    if (q0 == c1) continue;  // all key tiles in one cluster: it wrote the result
    // a lane reads the sums of parts lane and lane + 32 of the row, then all parts' outputs
    // come four at a time: read one after the other, a token of 128 heads over 8192 keys
    // (12 parts) took 9 us more
    const int parts = c1 - q0 + 1;
    float z[2], top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      z[i] = lane + 32 * i < parts ? __ldcg(lse_at(q0 + lane + 32 * i)) : -INFINITY;
      nan |= z[i] != z[i];
      top = fmaxf(top, z[i]);
    }
    nan = __any_sync(0xffffffffu, nan);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float acc[16] = {};
    float tot = 0.f;
    if (top != -INFINITY) {
#pragma unroll
      for (int i = 0; i < 2; ++i) z[i] = ex2((z[i] - top) * kLog2e);
      for (int i0 = 0; i0 < parts; i0 += 4) {
        float4 v[4][4];
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mine = i0 + i < 32 ? z[0] : z[1];
          w[i] = __shfl_sync(0xffffffffu, mine, (i0 + i) & 31);  // 0 behind the last part
          const int q = q0 + i0 + i;
          const float4* from = reinterpret_cast<const float4*>(p.part_out) +
                               part_at(2 * q + (a >= q * share ? 1 : 0), row & ~7) + 4 * (row & 7) + (lane & 3);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            v[i][y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (w[i] != 0.f) v[i][y] = __ldcg(from + 128 * (2 * y + (lane >> 4)) + 32 * ((lane >> 2) & 3));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tot += w[i];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            acc[4 * y] += w[i] * v[i][y].x;
            acc[4 * y + 1] += w[i] * v[i][y].y;
            acc[4 * y + 2] += w[i] * v[i][y].z;
            acc[4 * y + 3] += w[i] * v[i][y].w;
          }
        }
      }
    }
    const float inv = nan ? NAN : tot > 0.f ? 1.f / tot : 0.f;
    const int64_t to = tile.row0 + row;
    const int dim = 64 * (lane >> 4) + 32 * ((lane >> 3) & 1) + 8 * (lane & 3) + 4 * ((lane >> 2) & 1);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const float v0 = acc[4 * y] * inv, v1 = acc[4 * y + 1] * inv, v2 = acc[4 * y + 2] * inv,
                  v3 = acc[4 * y + 3] * inv;
      if (p.out_fp32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to * kLatent + 128 * y + dim) =
            make_float4(v0, v1, v2, v3);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to * kLatent + 128 * y + dim) =
            make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3));
    }
    if (lane == 0 && p.lse != nullptr)
      p.lse[to] = nan ? NAN : tot > 0.f ? top + lg2(tot) * kLn2 : -INFINITY;
  }
}

// ------------------------------------------------------------------ host
struct ChunkSpace {
  size_t tiles, first, failed, lse, out, bytes;  // offsets
  int32_t max_tiles;
};
ChunkSpace chunk_space(int32_t num_q, int32_t num_heads, int32_t num_seqs) {
  ChunkSpace s;
  const int64_t tiles =
      static_cast<int64_t>(num_q) * num_heads / kTileRows + (num_seqs < num_q ? num_seqs : num_q);
  s.max_tiles = static_cast<int32_t>(tiles);
  s.tiles = 64;
  s.first = s.tiles + sizeof(RowTile) * static_cast<size_t>(tiles);
  s.failed = s.first + 4 * kMaxClusters;
  s.lse = s.failed + 4 * kMaxClusters;
  s.out = s.lse + 4 * 2 * kMaxClusters * kTileRows;
  s.bytes = s.out + size_t{4} * 2 * kMaxClusters * kTileRows * kLatent;
  return s;
}
static_assert(kMaxClusters <= 64, "a lane of the merge has two parts");
static_assert(sizeof(RowTile) == 48 && sizeof(Plan) <= 64 && (4 * kMaxClusters) % 16 == 0, "workspace");

bool chunk_shape_ok(int32_t num_q, int32_t num_heads, int32_t num_seqs) {
  return num_q >= 0 && num_heads >= 1 && num_heads <= NVFP4_MLA_MAX_HEADS && num_seqs >= 1 &&
         num_seqs <= NVFP4_MLA_MAX_PLAN_SEQS &&
         static_cast<int64_t>(num_q) * num_heads <= INT32_MAX;
}

// Clusters of a kernel that the device holds at once, asked once a device.
template <int kFmt>
int32_t resident_clusters(int device, cudaLaunchConfig_t cfg, int sms, int* clusters) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int n = device < kDevices ? known[device].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 4 * 4));
    if (cudaOccupancyMaxActiveClusters(&n, chunk_kernel<kFmt>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return NVFP4_MLA_ERR_LAUNCH;
    }
    n = n < kMaxClusters ? n : kMaxClusters;
    if (device < kDevices) known[device].store(n, std::memory_order_relaxed);
  }
  *clusters = n;
  return NVFP4_MLA_OK;
}

template <int kFmt>
int32_t launch_chunk(ChunkParams p, int device, int sms, cudaStream_t stream) {
  constexpr size_t smem = ChunkLayout<kFmt>::kBytes;
  const size_t plan_smem = 4 * static_cast<size_t>(p.num_seqs);
  // limits of the process: the same in every call
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(chunk_kernel<kFmt>),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
      (plan_smem > 40 * 1024 &&
       cudaFuncSetAttribute(reinterpret_cast<const void*>(chunk_plan_kernel),
                            cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * NVFP4_MLA_MAX_PLAN_SEQS) != cudaSuccess)) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kChunkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  if (int32_t st = resident_clusters<kFmt>(device, cfg, sms, &p.clusters)) return st;
  if (p.invalid_count != nullptr) {
    chunk_check_kernel<<<p.num_seqs < 4 * sms ? p.num_seqs : 4 * sms, 256, 0, stream>>>(p);
    if (int32_t st = launch_status()) return st;
  }
  chunk_plan_kernel<<<1, kPlanThreads, plan_smem, stream>>>(p);
  if (int32_t st = launch_status()) return st;
  cfg.gridDim = dim3(static_cast<unsigned>(p.clusters * 4));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, chunk_kernel<kFmt>, p) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  cudaLaunchConfig_t last = {};
  last.gridDim = dim3(static_cast<unsigned>(4 * sms));
  last.blockDim = dim3(256);
  last.stream = stream;
  last.attrs = attr;
  last.numAttrs = 1;
  if (cudaLaunchKernelEx(&last, chunk_merge_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  return NVFP4_MLA_OK;
}

}  // namespace
}  // namespace nvfp4_mla

using namespace nvfp4_mla;

extern "C" size_t dense_mla_chunk_workspace_size(int32_t num_q, int32_t num_heads, int32_t num_seqs) {
  if (!chunk_shape_ok(num_q, num_heads, num_seqs)) return SIZE_MAX;
  return num_q == 0 ? 0 : chunk_space(num_q, num_heads, num_seqs).bytes;
}

extern "C" int32_t dense_mla_chunk(const void* q_latent, const void* q_rope, const int32_t* cu_tokens,
                                   int32_t num_q, int32_t num_heads, const int32_t* block_table,
                                   int32_t num_seqs, int32_t max_blocks_per_seq,
                                   const int32_t* seq_lens, int32_t page_size, const void* cache,
                                   int64_t num_blocks, int64_t block_stride_bytes, int32_t row_format,
                                   float sm_scale, float latent_scale, float rope_scale, void* out,
                                   int32_t out_fp32, float* lse, void* workspace,
                                   size_t workspace_bytes, int32_t* invalid_count, void* stream) {
  const int32_t rb = nvfp4_mla_row_bytes(row_format);
  if (rb == 0) return NVFP4_MLA_ERR_FORMAT;
  if (!chunk_shape_ok(num_q, num_heads, num_seqs)) return NVFP4_MLA_ERR_SHAPE;
  if (num_q == 0) return NVFP4_MLA_OK;
  if (!q_latent || !q_rope || !cu_tokens || !block_table || !seq_lens || !cache || !out)
    return NVFP4_MLA_ERR_NULL;
  if (max_blocks_per_seq <= 0 || page_size <= 0 || page_size > (1 << 20) ||
      static_cast<int64_t>(max_blocks_per_seq) * page_size > INT32_MAX - 511 || num_blocks <= 0 ||
      block_stride_bytes < static_cast<int64_t>(page_size) * rb ||
      block_stride_bytes > INT64_MAX / num_blocks)
    return NVFP4_MLA_ERR_SHAPE;
  if (!aligned16(q_latent) || !aligned16(q_rope) || !aligned16(cache) || !aligned16(out) ||
      (block_stride_bytes & 15))
    return NVFP4_MLA_ERR_ALIGN;
  if (!isfinite(sm_scale) || !(isfinite(rope_scale) && rope_scale > 0.f) ||
      !(isfinite(latent_scale) && latent_scale > 0.f))
    return NVFP4_MLA_ERR_VALUE;
  const ChunkSpace w = chunk_space(num_q, num_heads, num_seqs);
  if (!workspace || workspace_bytes < w.bytes) return NVFP4_MLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return NVFP4_MLA_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;

  ChunkParams p = {};
  p.q_lat = static_cast<const uint16_t*>(q_latent);
  p.q_rope = static_cast<const uint16_t*>(q_rope);
  p.cu_tokens = cu_tokens;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.num_q = num_q;
  p.num_heads = num_heads;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.page = page_division(page_size);
  p.cache = static_cast<const uint8_t*>(cache);
  p.num_blocks = num_blocks;
  p.block_stride = block_stride_bytes;
  const bool fp8 = row_format == NVFP4_MLA_ROW_FP8_576;
  const float lat = fp8 ? latent_scale : 1.f, sign = sm_scale < 0.f ? -1.f : 1.f;
  // never 0, so that the scale times -inf (a key that is not seen) stays -inf: times 2^-126 any
  // score of FP16 operands has an exponential of 1 too
  p.score_scale = fmaxf(fabsf(sm_scale) * lat * kLog2e, FLT_MIN);
  p.lat_mult = sign;
  p.rope_mult = sign * (rope_scale / lat);
  p.out_mult = lat;
  p.out = out;
  p.out_fp32 = out_fp32 ? 1 : 0;
  p.lse = lse;
  p.invalid_count = invalid_count;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<Plan*>(ws);
  p.tiles = reinterpret_cast<RowTile*>(ws + w.tiles);
  p.first = reinterpret_cast<int32_t*>(ws + w.first);
  p.failed = reinterpret_cast<int32_t*>(ws + w.failed);
  p.part_lse = reinterpret_cast<float*>(ws + w.lse);
  p.part_out = reinterpret_cast<float*>(ws + w.out);
  p.max_tiles = w.max_tiles;
  p.wait_cycles = decode_wait_cycles();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp8 ? launch_chunk<NVFP4_MLA_ROW_FP8_576>(p, dev, sms, s)
             : launch_chunk<NVFP4_MLA_ROW_NVFP4_352>(p, dev, sms, s);
}
