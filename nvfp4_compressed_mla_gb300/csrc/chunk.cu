// chunk.cu -- dense causal absorbed-MLA attention of a step's new tokens over the paged cache.
//
// Token i of the n new tokens of a sequence of length L sees keys 0 .. L - n + i. For each head
//   z_j = sm_scale (ql . lat_j + qr . rope_j),  out = sum_j softmax(z)_j lat_j,
// so keys and values are one row of the cache that all heads and tokens share: with M = (token,
// head) rows the step is two matrix products, S = Q K^T (576 deep) and O = P V (512 wide), with
// 2 x 1088 flop a row and key. A cache row of 352 bytes serves 128 heads with 279 kflop a token,
// 791 flop a byte: tensor-bound from one token of 128 heads on.
//
// The rows (token, head) of a sequence are consecutive in memory, and a tile takes 128 kPair of
// them, whatever the number of heads. One cluster works on a tile, and 512 columns of fp32 output
// for 128 rows are all of an SM's tensor memory, so that the two products live on different SMs:
//
//   score CTAs (ranks 0 .. kPair - 1): 128 rows each. Q stays in tensor memory (latent part, 256
//     columns, the MMA's A operand) and shared memory (rope part). Eight warps expand 64 keys a
//     CTA and tile into FP16 (exact: a code times its scale has 6 significant bits) in shared
//     memory; S of 64 kPair keys goes into one of two buffers. Four softmax warps (thread = row)
//     turn it into P = 2^(s c - m) against a lazy reference m, in FP16, and copy it in pieces of
//     64 keys into the output CTA of the same rows.
//   output CTAs (ranks kPair .. 2 kPair - 1): O (128 rows x 512, fp32) in tensor memory. Eight
//     warps expand the keys' latent part, each CTA 512 / kPair of the dimensions; four warps
//     (thread = row) rescale O when a row's reference moved, and write the output.
//
// With kPair = 2 each product is one MMA over a pair of SMs (cta_group::2, M = 256): an SM expands
// half of the keys or half of the dimensions and the pair shares them, which halves the work of
// expanding a key for a row. kPair = 1 wastes less on sequences with few rows.
//
// Work is dealt out in key tiles: a planning kernel lists the row tiles of the step with the key
// tiles that each sees, and every cluster takes an equal, contiguous share of all of them. A row
// tile that is cut by the shares' borders is merged by a last kernel from fp32 partial results.
//
// Every wait is bounded. A cluster whose wait runs out drains what it has in flight and reports
// it; the last kernel then writes NaN to all rows of the step.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "decode_common.cuh"
#include "plan_common.cuh"
#include "tc_ptx.cuh"

namespace nvfp4_mla {
namespace {

constexpr int kPieceKeys = 64;                // keys of a P piece and of a V slot
constexpr int kSoftWarps = 8;                 // softmax / rescaling and output: two groups of four
constexpr int kExpandWarp0 = 8, kExpandWarps = 8;
constexpr int kIssueWarp = 16, kSendWarp = 17;
constexpr int kChunkThreads = 20 * 32;        // the last four warps leave registers to the others
// Registers of a thread of the softmax, the expanding and the last warps; as
// many in all as at the launch.
constexpr int kSoftRegs = 112, kExpandRegs = 112, kIssueRegs = 32;
static_assert(2 * kSoftRegs + 2 * kExpandRegs + kIssueRegs == 5 * 96, "registers");
constexpr int kMaxClusters = 80;              // of two CTAs; half as many of four
constexpr int kPSlots = 4;                    // P pieces in flight
constexpr uint32_t kPBytes = 128 * kPieceKeys * 2;
constexpr uint32_t kKBlock = kPieceKeys * 128;   // 64 keys x 64 dimensions, FP16
constexpr uint32_t kKTileBytes = 9 * kKBlock;    // 8 latent blocks and the rope
constexpr long long kDrainLimit = 1ll << 31;
// The reference of a row moves when a score exceeds it by more than kTau (log2
// units), to kHeadroom below that score. P <= 2^15 fits FP16 (largest finite
// value 65504) and P of the largest score is at least 2^kHeadroom then, so that
// weights down to 2^-21 of it are normal FP16 numbers.
constexpr float kTau = 15.f, kHeadroom = 7.f;
// Key tiles' time that a row tile costs beside its own (loading Q, the first
// score tile before P V can begin, writing O), and the least share of a cluster.
template <int kPair> constexpr int kTileOverhead = kPair == 2 ? 3 : 6;
template <int kPair> constexpr int kLeastShare = kPair == 2 ? 6 : 12;

struct RowTile {       // 128 kPair rows of a sequence
  int32_t seq, index;  // of the sequence's row tiles
  int64_t unit;        // first unit: kTileOverhead units, then one a key tile
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
  RowTile* tiles;     // [max_tiles + 1]
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
template <int kPair>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p) {
  extern __shared__ int32_t upto[];  // [num_seqs] row tiles up to and with sequence s
  __shared__ int64_t sums[32];
  constexpr int kRows = 128 * kPair, kKeys = kPieceKeys * kPair;
  cudaTriggerProgrammaticLaunchCompletion();
  const int tid = threadIdx.x;
  int64_t tiles = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int32_t start, len;
    const int64_t rows =
        s < p.num_seqs ? static_cast<int64_t>(new_tokens(p, s, start, len)) * p.num_heads : 0;
    const int64_t to = block_scan((rows + kRows - 1) / kRows, tiles, sums);
    // offsets that overlap could ask for more than there is room for
    if (s < p.num_seqs) upto[s] = static_cast<int32_t>(min(to, static_cast<int64_t>(p.max_tiles)));
  }
  const int32_t n_tiles = static_cast<int32_t>(min(tiles, static_cast<int64_t>(p.max_tiles)));
  __syncthreads();
  int64_t units = 0;
  for (int t0 = 0; t0 < n_tiles; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int64_t n = 0;
    int s = 0, index = 0;
    if (t < n_tiles) {
      int hi = p.num_seqs - 1;
      while (s < hi) {
        const int mid = (s + hi) >> 1;
        if (upto[mid] <= t) s = mid + 1;
        else hi = mid;
      }
      index = t - (s > 0 ? upto[s - 1] : 0);
      int32_t start, len;
      const int32_t tokens = new_tokens(p, s, start, len);
      const int64_t last = min((static_cast<int64_t>(index) * kRows + kRows - 1) / p.num_heads,
                               static_cast<int64_t>(tokens - 1));
      n = kTileOverhead<kPair> + (len - tokens + last + kKeys) / kKeys;  // sees len - tokens + last + 1
    }
    const int64_t to = block_scan(n, units, sums);
    if (t < n_tiles) p.tiles[t] = {s, index, to - n};
  }
  const int64_t share = max((units + p.clusters - 1) / p.clusters, int64_t{kLeastShare<kPair>});
  for (int c = tid; c < p.clusters; c += kPlanThreads) {
    p.first[c] = n_tiles;
    p.failed[c] = 0;
  }
  if (tid == 0) {
    p.tiles[n_tiles] = {-1, 0, units};
    *p.plan = {units, share, n_tiles, 0};
  }
  __syncthreads();
  for (int t = tid; t < n_tiles; t += kPlanThreads) {
    const int64_t a = p.tiles[t].unit, b = p.tiles[t + 1].unit;
    for (int64_t c = (a + share - 1) / share; c * share < b; ++c) p.first[c] = t;
  }
}

// Positions without a page, and malformed sequences; launched where they are counted.
__global__ void __launch_bounds__(256) chunk_check_kernel(const ChunkParams p) {
  int bad = 0;
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
  if (bad > 0) atomicAdd(p.invalid_count, bad);
}

// The pieces of row tiles that make up a cluster's share, one after the other.
template <int kPair>
struct Pieces {
  const ChunkParams& p;
  int64_t u0, u1;     // the cluster's units
  int32_t t, tiles;   // the next row tile
  int32_t cluster;
  // the current piece
  int32_t seq, rows, base, len;  // rows of the tile; tokens before the new ones; length
  int64_t row0, first_row;       // first row of the tile, of the sequence's first token
  int32_t begin, end;            // key tiles
  bool whole;                    // all that the row tile sees
  int32_t slot;                  // of a partial result

  __device__ Pieces(const ChunkParams& params, int c) : p(params), cluster(c) {
    const int64_t units = __ldcg(&p.plan->units), share = __ldcg(&p.plan->share);
    u0 = c * share;
    u1 = min(u0 + share, units);
    tiles = __ldcg(&p.plan->tiles);
    t = u0 < units ? __ldcg(p.first + c) : tiles;
  }
  __device__ __forceinline__ bool next() {
    while (t < tiles) {
      const int4 x = __ldcg(reinterpret_cast<const int4*>(p.tiles + t));
      const int4 y = __ldcg(reinterpret_cast<const int4*>(p.tiles + t + 1));
      const int64_t a = static_cast<int64_t>(static_cast<uint32_t>(x.z)) | (static_cast<int64_t>(x.w) << 32);
      const int64_t b = static_cast<int64_t>(static_cast<uint32_t>(y.z)) | (static_cast<int64_t>(y.w) << 32);
      if (a >= u1) break;
      ++t;
      const int64_t k0 = a + kTileOverhead<kPair>;  // unit of key tile 0
      begin = static_cast<int32_t>(max(u0 - k0, int64_t{0}));
      end = static_cast<int32_t>(max(min(u1, b) - k0, int64_t{0}));
      if (end <= begin) continue;
      whole = begin == 0 && end == b - k0;
      slot = 2 * cluster + (a >= u0 ? 1 : 0);
      seq = x.x;
      int32_t start;
      const int32_t n = new_tokens(p, seq, start, len);
      base = len - n;
      first_row = static_cast<int64_t>(start) * p.num_heads;
      row0 = first_row + static_cast<int64_t>(x.y) * (128 * kPair);
      rows = static_cast<int32_t>(
          min(static_cast<int64_t>(n) * p.num_heads - (row0 - first_row), int64_t{128 * kPair}));
      return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void arrive_tx_release_cluster(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cluster.shared::cluster.b64 _, [%0], %1;" ::
                   "r"(cluster_bar),
               "r"(bytes)
               : "memory");
}
// The same where only copied bytes are to be seen behind the barrier.
__device__ __forceinline__ void arrive_tx_relaxed_cluster(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::
                   "r"(cluster_bar),
               "r"(bytes)
               : "memory");
}
// shared (this CTA) -> shared (another CTA of the cluster), counted on that CTA's mbarrier
__device__ __forceinline__ void bulk_s2s(uint32_t dst_cluster, uint32_t src, uint32_t bytes,
                                         uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst_cluster),
      "r"(src), "r"(bytes), "r"(bar_cluster)
      : "memory");
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kPair>
__device__ __forceinline__ void alloc_tmem(uint32_t dst_smem) {
  if constexpr (kPair == 1) {
    tmem_alloc(dst_smem);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int kPair>
__device__ __forceinline__ void free_tmem(uint32_t taddr) {
  if constexpr (kPair == 1) {
    tmem_dealloc(taddr);
  } else {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                 "r"(kTmemCols)
                 : "memory");
  }
}
template <int kPair>
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  if constexpr (kPair == 1) {
    mma_ss(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
template <int kPair>
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  if constexpr (kPair == 1) {
    mma_ts(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// One arrival on the barrier at this offset in every CTA of `mask`, once all
// MMAs that this thread issued before have completed.
template <int kPair>
__device__ __forceinline__ void commit_to(uint32_t bar, uint16_t mask) {
  if constexpr (kPair == 1)
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"(mask)
        : "memory");
  else
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
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort_addr,
                                          long long limit) {
  return __all_sync(0xffffffffu, wait_bar_hot<kCluster>(bar, parity, abort_addr, limit));
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
__device__ __forceinline__ uint4 ld_row_v4(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint32_t ld_row_u16(const uint8_t* p) {
  uint16_t r;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(r) : "l"(p));
  return r;
}
__device__ __forceinline__ uint4 to_f16x8(uint4 x, float m) {  // 8 bf16 values times m
  return make_uint4(pack_f16x2(bf16_lo(x.x) * m, bf16_hi(x.x) * m),
                    pack_f16x2(bf16_lo(x.y) * m, bf16_hi(x.y) * m),
                    pack_f16x2(bf16_lo(x.z) * m, bf16_hi(x.z) * m),
                    pack_f16x2(bf16_lo(x.w) * m, bf16_hi(x.w) * m));
}

// ------------------------------------------------------------------ memory plan
template <int kPair>
struct ChunkLayout {
  // score CTA
  static constexpr uint32_t kK = 0;                        // two key tiles
  static constexpr uint32_t kQRope = 2 * kKTileBytes;
  static constexpr uint32_t kStaged = kQRope + 16384;      // P pieces on their way out
  static constexpr uint32_t kRef = kStaged + kPSlots * kPBytes;  // references of the rows, two pieces
  static constexpr uint32_t kSums = kRef + 1024;                 // sums of weights, two results
  static constexpr uint32_t kEndScore = kSums + 1024;
  // output CTA
  static constexpr uint32_t kVSlot = 65536 / kPair;        // 64 keys x 512 / kPair dimensions
  static constexpr int kVSlots = 2 * kPair;
  static constexpr uint32_t kV = 0;
  static constexpr uint32_t kP = kV + kVSlots * kVSlot;
  static constexpr uint32_t kFactor = kP + kPSlots * kPBytes;  // rescale factor of each row, a P slot
  static constexpr uint32_t kTag = kFactor + kPSlots * 512;    // per warp and P slot: 1 + piece to rescale at
  static constexpr uint32_t kFinal = kTag + kPSlots * 16;      // output factor of each row, a result
  static constexpr uint32_t kFinals = 8;  // more results than there are P pieces in flight
  static constexpr uint32_t kEndOut = kFinal + kFinals * 512;
  static constexpr uint32_t kCtl = kEndScore > kEndOut ? kEndScore : kEndOut;
  static constexpr uint32_t kCtlBytes = 1024;
  static constexpr uint32_t kBytes = kCtl + kCtlBytes;
  // score CTA's tensor memory: Q's latent part in columns 0 .. 255, then S
  static constexpr uint32_t kSCol = 256;
  static constexpr uint32_t kSBufs = 4 / kPair;
  static_assert(kBytes <= kMaxSharedBytes && kCtl % 16 == 0, "shared memory");
  static_assert(kSCol + kSBufs * kPieceKeys * kPair <= kTmemCols, "tensor memory");
};
struct ChunkCtl {  // barriers and words, at the same offsets in every CTA of the cluster
  static constexpr uint32_t kKFull = 0, kSFull = 16, kSEmpty = 48, kQFull = 80, kPFull = 88,
                            kPReady = 136, kVFull = 184, kPvDone = 216, kTask = 264, kTaskDone = 272,
                            kStaged = 280, kRefDone = 328, kSumDone = 392, kTmem = 456, kAbort = 460,
                            kSent = 464, kScored = 468, kSummed = 472, kTaskWord = 476, kNoted = 480,
                            kMissing = 512;
  // a word for each of the expanding warps of a tile, 8 tiles: (1 + tile) << 8 and
  // the bits of its keys that exist, where some page does not resolve
  static constexpr uint32_t kMissingTiles = 8, kMissingBytes = 64;
};
static_assert(kPSlots <= 6 && ChunkCtl::kNoted + 4 * kPSlots <= ChunkCtl::kMissing &&
                  ChunkCtl::kMissing + 512 == ChunkLayout<1>::kCtlBytes,
              "control block");

// ------------------------------------------------------------------ expansion
// Warp w of the eight expands keys 8 w .. 8 w + 7 of each 64. kItems 16-byte
// pieces of cache rows a lane, in registers from their load on:
//   NVFP4 rows: 32 codes (64 bytes of FP16) and their two scales; a lane has two
//     keys, (lane / 2) % 4 and that + 4; rope: key lane / 4, bytes 16 (lane % 4);
//   FP8 rows: 16 values of key lane / 4.
// Both ways the eight lanes of a store's phase write eight different 16-byte
// columns of the swizzled 128-byte rows.
template <int kFmt, int kLatItems, bool kRopeToo>
struct RowItems {
  static constexpr bool kNv = kFmt == NVFP4_MLA_ROW_NVFP4_352;
  uint4 lat[kLatItems];
  uint32_t scale[kNv ? kLatItems : 1];
  uint4 rope;
};

// Where a lane's first latent item lies from the warp's first key on, in bytes.
// An output CTA of a pair (kHalves) expands dimensions 128 part .. + 127 of each
// half of the 512.
template <int kFmt, bool kHalves>
__device__ __forceinline__ uint32_t first_item(int lane, int part) {
  if constexpr (kFmt == NVFP4_MLA_ROW_NVFP4_352) {
    const uint32_t c = (lane & 1) + 2 * (lane >> 3);  // 32 dimensions each
    return ((lane >> 1) & 3) * kNvfp4Row + (kHalves ? 128 * (c >> 2) + 64 * part + 16 * (c & 3) : 16 * c);
  } else {
    return (lane >> 2) * kFp8Row + (kHalves ? 128 * part : 0) + 16 * (lane & 3);
  }
}
// The distance from there to item i, and (NVFP4) the distance of its two scales.
template <int kFmt, bool kHalves>
__device__ __forceinline__ constexpr uint32_t item_step(int i) {
  if (kFmt == NVFP4_MLA_ROW_NVFP4_352) return (i & 1) * 4 * kNvfp4Row + (i >> 1) * 128;
  return kHalves ? 256 * (i >> 1) + 64 * (i & 1) : 64 * i;
}
__device__ __forceinline__ constexpr uint32_t scale_step(int i) {
  return (i & 1) * 4 * kNvfp4Row + (i >> 1) * 16;
}
__device__ __forceinline__ uint32_t first_scale(uint32_t item) {  // of the item at this distance
  const uint32_t key = item / kNvfp4Row;
  return key * kNvfp4Row + kScaleOff + (item - key * kNvfp4Row) / 8;
}
template <int kFmt>
__device__ __forceinline__ uint32_t rope_item(int lane) {
  return kFmt == NVFP4_MLA_ROW_NVFP4_352 ? (lane >> 2) * kNvfp4Row + kRopeOff + 16 * (lane & 3)
                                         : (lane >> 2) * kFp8Row + kLatent + 16 * (lane & 3);
}

// The keys of a warp at a time: where the first one lies, or all eight.
// kRuns (pages of a multiple of 64 rows): one page holds them, and a lane's items
// lie at fixed distances; rows of the page behind the length are read as they
// are (no row sees them, and as values they are numbers). Otherwise lane j has
// the address of key j.
template <int kFmt, bool kRuns, bool kHalves>
struct KeyRows {
  static constexpr int kRowBytes = kFmt == NVFP4_MLA_ROW_NVFP4_352 ? kNvfp4Row : kFp8Row;
  uint32_t lat0, scale0, rope0;  // of the lane, from the warp's first key on
  int part;
  int32_t page, in_page;  // of the next keys: the entry is on its way
  bool some;              // they are below the length

  __device__ KeyRows(int lane, int part_) : part(part_) {
    lat0 = first_item<kFmt, kHalves>(lane, part);
    scale0 = first_scale(lat0);
    rope0 = rope_item<kFmt>(lane);
  }
  __device__ __forceinline__ void none() {
    page = -1;
    some = false;
  }
  // the entry of keys first_key + 8 w .. + 7 of 64, on its way
  __device__ __forceinline__ void next(const ChunkParams& p, int32_t seq, int32_t first_key, int w, int32_t len,
                                       int lane) {
    const int32_t key = first_key + (kRuns ? 0 : 8 * w + (lane & 7));
    some = key < len && (kRuns || lane < 8);
    page = -1;
    if (some) {
      const int32_t b = p.page.block(key);
      in_page = key - b * p.page.size + (kRuns ? 8 * w : 0);
      page = __ldg(p.block_table + static_cast<int64_t>(seq) * p.max_blocks + b);
    }
  }
  // loads them; `exist` and `missing` are bits of the eight keys
  template <int kLatItems, bool kRopeToo>
  __device__ __forceinline__ void load(const ChunkParams& p, int lane, RowItems<kFmt, kLatItems, kRopeToo>& r,
                                       uint32_t& exist, uint32_t& missing) const {
    using R = RowItems<kFmt, kLatItems, kRopeToo>;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const bool ok = page >= 0 && page < p.num_blocks;
    const int64_t mine = page * p.block_stride + static_cast<int64_t>(in_page) * kRowBytes;
    if constexpr (kRuns) {
      exist = ok ? 0xffu : 0u;
      missing = some && !ok ? 0xffu : 0u;
      const uint8_t* lat = p.cache + mine + lat0;
      if (ok) {
#pragma unroll
        for (int i = 0; i < kLatItems; ++i) r.lat[i] = ld_row_v4(lat + item_step<kFmt, kHalves>(i));
        if constexpr (R::kNv) {
          const uint8_t* sc = p.cache + mine + scale0;
#pragma unroll
          for (int i = 0; i < kLatItems; ++i) r.scale[i] = ld_row_u16(sc + scale_step(i));
        }
        if constexpr (kRopeToo) r.rope = ld_row_v4(p.cache + mine + rope0);
      } else {
#pragma unroll
        for (int i = 0; i < kLatItems; ++i) r.lat[i] = z;
        if constexpr (R::kNv) {
#pragma unroll
          for (int i = 0; i < kLatItems; ++i) r.scale[i] = 0u;
        }
        if constexpr (kRopeToo) r.rope = z;
      }
    } else {
      exist = __ballot_sync(0xffffffffu, ok);
      missing = __ballot_sync(0xffffffffu, some && !ok);
      const int64_t off = ok ? mine : -1;
      const uint32_t key0 = lat0 / kRowBytes;  // of the lane's items; the same for the scales
      const uint32_t in_row = lat0 - key0 * kRowBytes, scale_in_row = scale0 - key0 * kRowBytes;
      const int64_t at[2] = {__shfl_sync(0xffffffffu, off, key0),
                             R::kNv ? __shfl_sync(0xffffffffu, off, (key0 + 4) & 31) : 0};
#pragma unroll
      for (int i = 0; i < kLatItems; ++i) {
        const int64_t a = at[R::kNv ? i & 1 : 0];
        const uint32_t step = item_step<kFmt, kHalves>(i) - (R::kNv ? (i & 1) * 4 * kNvfp4Row : 0);
        r.lat[i] = a >= 0 ? ld_row_v4(p.cache + a + in_row + step) : z;
        if constexpr (R::kNv)
          r.scale[i] = a >= 0 ? ld_row_u16(p.cache + a + scale_in_row + (scale_step(i) - (i & 1) * 4 * kNvfp4Row)) : 0u;
      }
      if constexpr (kRopeToo) {
        const int64_t a = __shfl_sync(0xffffffffu, off, lane >> 2);
        r.rope = a >= 0 ? ld_row_v4(p.cache + a + (rope0 - (lane >> 2) * kRowBytes)) : z;
      }
    }
  }
};

__device__ __forceinline__ void store_e4m3x16(uint4 v, uint32_t block, uint32_t key, uint32_t col,
                                              bool numbers) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    h[2 * q] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[q] & 0xFFFFu));
    h[2 * q + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[q] >> 16));
  }
  if (numbers) {
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = hmin2(h[q], 0x5F005F00u);  // 448
  }
  st_shared_v4(block + swizzled(key, col), h[0], h[1], h[2], h[3]);
  st_shared_v4(block + swizzled(key, col + 1), h[4], h[5], h[6], h[7]);
}

// Into blocks of 64 keys x 64 dimensions from `dst` on. `kNumbers` (the output
// CTAs): a NaN in a row becomes a number. Its scores are NaN for every token that
// sees the row; the others weigh it with 0, which a NaN would not survive.
template <int kFmt, int kLatItems, bool kRopeToo, bool kNumbers>
__device__ __forceinline__ void store_items(const RowItems<kFmt, kLatItems, kRopeToo>& r, uint32_t dst,
                                            int warp, int lane) {
  using R = RowItems<kFmt, kLatItems, kRopeToo>;
  if constexpr (R::kNv) {
#pragma unroll
    for (int i = 0; i < kLatItems; ++i) {
      const uint32_t key = 8u * warp + ((lane >> 1) & 3) + 4u * (i & 1);
      const uint32_t c = (lane & 1) + 2 * (lane >> 3) + 8 * (i >> 1);
      uint32_t s = e4m3x2_to_f16x2(static_cast<uint16_t>(r.scale[i]));
      if (kNumbers) s = hmin2(s, 0x5F005F00u);
      const uint32_t s0 = __byte_perm(s, s, 0x1010), s1 = __byte_perm(s, s, 0x3232);
      const uint32_t w[4] = {r.lat[i].x, r.lat[i].y, r.lat[i].z, r.lat[i].w};
      const uint32_t block = dst + (c >> 1) * kKBlock;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t f[4];
        e2m1x8_to_f16x8(w[x], f);
#pragma unroll
        for (int y = 0; y < 4; ++y) f[y] = hmul2_u32(f[y], x < 2 ? s0 : s1);
        st_shared_v4(block + swizzled(key, (c & 1) * 4 + x), f[0], f[1], f[2], f[3]);
      }
    }
  } else {
    const uint32_t key = 8u * warp + (lane >> 2);
#pragma unroll
    for (int i = 0; i < kLatItems; ++i) {
      const uint32_t c = 4 * i + (lane & 3);
      store_e4m3x16(r.lat[i], dst + (c >> 2) * kKBlock, key, 2 * (c & 3), kNumbers);
    }
  }
  if constexpr (kRopeToo)
    store_e4m3x16(r.rope, dst + 8 * kKBlock, 8u * warp + (lane >> 2), 2 * (lane & 3), false);
}

// A walk over the units of keys of a cluster's pieces: key tiles (score CTAs)
// or pieces of 64 keys (output CTAs).
template <int kPair>
struct KeyWalk {
  Pieces<kPair> pieces;
  int32_t at, end;  // in steps of the walk
  int32_t per;      // steps a key tile
  bool live;
  __device__ KeyWalk(const ChunkParams& p, int cluster, int steps) : pieces(p, cluster), per(steps) {
    start();
  }
  __device__ __forceinline__ void start() {
    live = pieces.next();
    at = live ? pieces.begin * per : 0;
    end = live ? pieces.end * per : 0;
  }
  __device__ __forceinline__ void step() {
    if (++at == end) start();
  }
};

// ------------------------------------------------------------------ kernel
template <int kFmt, int kPair, bool kRuns>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(const ChunkParams p) {
  using L = ChunkLayout<kPair>;
  using C = ChunkCtl;
  constexpr bool kNv = kFmt == NVFP4_MLA_ROW_NVFP4_352;
  constexpr int kTileKeys = kPieceKeys * kPair;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ctl = sbase + L::kCtl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = static_cast<int>(blockIdx.x) / (2 * kPair);
  const bool scoring = rank < kPair;
  const uint32_t part = scoring ? rank : rank - kPair;  // which of the pair
  const uint32_t leader = scoring ? 0 : kPair;
  const long long lim = p.wait_cycles;
  const uint32_t abort_addr = ctl + C::kAbort;
  auto bar = [&](uint32_t off, uint32_t i) { return ctl + off + 8u * i; };
  // an arrival at the leader of this CTA's pair, behind this thread's writes
  const uint32_t leader_ctl = map_rank(ctl, leader);
  auto tell_leader = [&](uint32_t off, uint32_t i) {
    if constexpr (kPair == 1) mbar_arrive(bar(off, i));
    else mbar_arrive_cluster(leader_ctl + off + 8u * i);
  };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(bar(C::kKFull, i), kExpandWarps * kPair);
    for (uint32_t i = 0; i < L::kSBufs; ++i) {
      mbar_init(bar(C::kSFull, i), 1);
      mbar_init(bar(C::kSEmpty, i), 4 * kPair * kPair);  // the warps that read a tile, of each CTA
    }
    mbar_init(bar(C::kQFull, 0), kSoftWarps * kPair);
    for (int i = 0; i < kPSlots; ++i) {
      mbar_init(bar(C::kPFull, i), 1);
      mbar_init(bar(C::kPReady, i), 1);
      mbar_init(bar(C::kPvDone, i), 1);
      mbar_init(bar(C::kStaged, i), 4);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(bar(C::kRefDone, i), 1);
      mbar_init(bar(C::kSumDone, i), 1);
    }
    for (int i = 0; i < L::kVSlots; ++i) mbar_init(bar(C::kVFull, i), kExpandWarps * kPair);
    mbar_init(bar(C::kTask, 0), 1);
    mbar_init(bar(C::kTaskDone, 0), kSoftWarps);
    st_shared_u32(ctl + C::kSent, 0u);
    st_shared_u32(ctl + C::kScored, 0u);
    st_shared_u32(ctl + C::kSummed, 0u);
    for (int i = 0; i < kPSlots; ++i) st_shared_u32(ctl + C::kNoted + 4 * i, 0u);
    st_shared_u32(abort_addr, (sbase & 1023u) != 0 ? 1u : 0u);
    fence_mbar_init();
  }
  if (tid < 128) st_shared_u32(ctl + C::kMissing + 4 * tid, 0u);
  if (!scoring && tid < 4 * kPSlots) st_shared_u32(sbase + L::kTag + 4 * tid, 0u);
  if (warp == kIssueWarp) alloc_tmem<kPair>(ctl + C::kTmem);
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
    fewer_registers<kIssueRegs>();
    if (warp == kSendWarp && scoring) {
      // ------------------------------------------------ P pieces to the output CTA
      if (lane == 0) {
        const uint32_t out_rank = kPair + part;
        const uint32_t out_p = map_rank(sbase + L::kP, out_rank), out_full = map_rank(bar(C::kPFull, 0), out_rank);
        uint32_t u = 0;
        bool run = true;
        Pieces<kPair> pieces(p, cluster);
        while (run && pieces.next()) {
          const uint32_t n = static_cast<uint32_t>(pieces.end - pieces.begin) * kPair;
          for (uint32_t x = 0; x < n; ++x, ++u) {
            const uint32_t ps = u % kPSlots;
            run = wait_bar_hot(bar(C::kStaged, ps), (u / kPSlots) & 1, abort_addr, lim);
            if (!run) break;
            const uint32_t full = out_full + 8u * ps;
            if (ld_shared_u32(ctl + C::kNoted + 4 * ps) == u + 1) arrive_tx_release_cluster(full, kPBytes);
            else arrive_tx_relaxed_cluster(full, kPBytes);
            bulk_s2s(out_p + ps * kPBytes, sbase + L::kStaged + ps * kPBytes, kPBytes, full);
          }
        }
        st_cluster_u32(map_rank(ctl + C::kSent, out_rank), u);
      }
    } else if (warp == kIssueWarp && scoring) {
      // ------------------------------------------------ S = Q K^T (one thread of the leader)
      if (lane == 0 && rank == leader) {
        constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(kTileKeys >> 3) << 17) |
                                    (static_cast<uint32_t>(128 * kPair >> 4) << 24);
        const uint64_t qr = operand_desc(sbase + L::kQRope);
        uint32_t i = 0;
        bool run = true;
        Pieces<kPair> pieces(p, cluster);
        for (uint32_t item = 0; run && pieces.next(); ++item) {
          if (!wait_bar_hot<true>(bar(C::kQFull, 0), item & 1, abort_addr, lim)) break;
          for (int32_t kt = pieces.begin; kt < pieces.end; ++kt, ++i) {
            const uint32_t b = i % L::kSBufs, slot = i & 1;
            if (!wait_bar_hot<true>(bar(C::kSEmpty, b), ((i / L::kSBufs) & 1) ^ 1, abort_addr, lim) ||
                !wait_bar_hot<true>(bar(C::kKFull, slot), (i >> 1) & 1, abort_addr, lim)) {
              run = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = L::kSCol + kTileKeys * b;
            const uint64_t kd = operand_desc(sbase + L::kK + slot * kKTileBytes);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              pair_mma_ts<kPair>(d, 8u * x, kd + (x >> 2) * (kKBlock >> 4) + 2 * (x & 3), kIdesc,
                                 x != 0 ? 1u : 0u);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              pair_mma_ss<kPair>(d, qr + 2 * x, kd + 8 * (kKBlock >> 4) + 2 * x, kIdesc, 1u);
            commit_to<kPair>(bar(C::kSFull, b), static_cast<uint16_t>((1u << kPair) - 1));
          }
        }
        for (uint32_t r = 0; r < kPair; ++r) st_cluster_u32(map_rank(ctl + C::kScored, r), i);
      }
    } else if (warp == kIssueWarp) {
      // ------------------------------------------------ O += P V (one thread of the leader)
      // A thread of each output CTA follows the P pieces that land there. It has O
      // rescaled where a piece comes with factors and written behind the last piece
      // of a row tile (tasks of warps 0-3), then the leader's issues the MMAs and the
      // other one tells it that its piece is there.
      if (lane == 0) {
        constexpr uint32_t kIdesc = (1u << 4) | (1u << 16) | ((256u >> 3) << 17) |
                                    (static_cast<uint32_t>(128 * kPair >> 4) << 24);
        uint32_t u = 0, tasks = 0;
        bool run = true;
        auto post = [&](uint32_t word) {
          st_shared_u32(ctl + C::kTaskWord, word);
          mbar_arrive(bar(C::kTask, 0));
          ++tasks;
        };
        auto task_done = [&]() { return wait_bar_hot(bar(C::kTaskDone, 0), (tasks - 1) & 1, abort_addr, lim); };
        Pieces<kPair> pieces(p, cluster);
        while (run && pieces.next()) {
          const uint32_t n = static_cast<uint32_t>(pieces.end - pieces.begin) * kPair;
          if (tasks > 0 && !task_done()) break;  // O before has been read
          for (uint32_t x = 0; x < n; ++x, ++u) {
            const uint32_t ps = u % kPSlots, vs = u % L::kVSlots;
            run = wait_bar_hot<true>(bar(C::kPFull, ps), (u / kPSlots) & 1, abort_addr, lim);
            if (!run) break;
            const uint4 tag = ld_shared_v4(sbase + L::kTag + 16 * ps);
            if (tag.x == u + 1 || tag.y == u + 1 || tag.z == u + 1 || tag.w == u + 1) {
              post(2 * u);
              run = task_done();
              if (!run) break;
            }
            tc_fence_after();
            if (rank != leader) {
              tc_fence_before();
              mbar_arrive_cluster(map_rank(bar(C::kPReady, ps), leader));
              continue;
            }
            run = (kPair == 1 || wait_bar_hot<true>(bar(C::kPReady, ps), (u / kPSlots) & 1, abort_addr, lim)) &&
                  wait_bar_hot<true>(bar(C::kVFull, vs), (u / L::kVSlots) & 1, abort_addr, lim);
            if (!run) break;
            tc_fence_after();
            const uint64_t pd = operand_desc(sbase + L::kP + ps * kPBytes);
            const uint64_t vd = operand_desc(sbase + L::kV + vs * L::kVSlot, kKBlock);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int nh = 0; nh < 2; ++nh)
                pair_mma_ss<kPair>(256u * nh, pd + 2 * kk,
                                   vd + nh * (L::kVSlot >> 5) + kk * (2048 >> 4), kIdesc,
                                   (x | kk) != 0 ? 1u : 0u);
            commit_to<kPair>(bar(C::kPvDone, ps), static_cast<uint16_t>((1u << (2 * kPair)) - 1));
          }
          if (run) post(2 * (u - 1) + 1);
        }
        if (rank == leader)
          for (uint32_t r = 0; r < 2 * kPair; ++r) st_cluster_u32(map_rank(ctl + C::kSummed, r), u);
      }
    }
  } else if (warp >= kExpandWarp0) {
    more_registers<kExpandRegs>();
    if (scoring) {
      // ------------------------------------------------ keys of a score CTA
      // Tile i goes into slot i % 2, once the MMAs of tile i - 2 are done. Rows are
      // loaded kAhead tiles ahead and table entries one more; the loop is unrolled
      // over the kAhead + 1 sets of registers, so that no copy waits for a load.
      constexpr int kLat = kNv ? 4 : 8, kAhead = kNv ? 2 : 1, kSets = kAhead + 1;
      using R = RowItems<kFmt, kLat, true>;
      const int w = warp - kExpandWarp0;
      KeyWalk<kPair> walk(p, cluster, 1);
      KeyRows<kFmt, kRuns, false> rows(lane, 0);
      auto entry = [&]() {
        if (!walk.live) {
          rows.none();
          return;
        }
        rows.next(p, walk.pieces.seq, walk.at * kTileKeys + kPieceKeys * static_cast<int32_t>(part), w,
                  walk.pieces.len, lane);
        walk.step();
      };
      R items[kSets];
      uint32_t exist[kSets], missing[kSets];  // bits of the warp's keys
      bool live[kSets];
      bool next_live = walk.live;
      entry();
      auto fetch = [&](int k) {  // rows into set k, and the next table entry
        live[k] = next_live;
        rows.load(p, lane, items[k], exist[k], missing[k]);
        next_live = walk.live;
        entry();
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k) fetch(k);
      bool run = true;
      for (uint32_t i = 0; run;) {
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
          if (!run || !live[k]) {
            run = false;
            break;
          }
          fetch((k + kAhead) % kSets);
          if (i >= 2 && !warp_wait(bar(C::kSFull, (i - 2) % L::kSBufs), ((i - 2) / L::kSBufs) & 1, abort_addr, lim)) {
            run = false;
            break;
          }
          store_items<kFmt, kLat, true, false>(items[k], sbase + L::kK + (i & 1) * kKTileBytes, w, lane);
          fence_proxy_async_cta();
          if (missing[k] != 0u) {  // the softmax of both CTAs has to know
            if (lane < kPair)
              st_cluster_u32(map_rank(ctl + C::kMissing + C::kMissingBytes * (i % C::kMissingTiles) + 4 * (8 * part + w), lane),
                             ((i + 1) << 8) | exist[k]);
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) tell_leader(C::kKFull, i & 1);
          ++i;
        }
      }
    } else {
      // ------------------------------------------------ values of an output CTA
      // Piece u goes into slot u % kVSlots, once the MMAs of piece u - kVSlots are done.
      constexpr int kLat = (kNv ? 4 : 8) / kPair, kAhead = kLat > 4 ? 1 : 2, kSets = kAhead + 1;
      using R = RowItems<kFmt, kLat, false>;
      const int w = warp - kExpandWarp0;
      KeyWalk<kPair> walk(p, cluster, kPair);
      KeyRows<kFmt, kRuns, kPair == 2> rows(lane, static_cast<int>(part));
      auto entry = [&]() {
        if (!walk.live) {
          rows.none();
          return;
        }
        rows.next(p, walk.pieces.seq, walk.at * kPieceKeys, w, walk.pieces.len, lane);
        walk.step();
      };
      R items[kSets];
      bool live[kSets];
      bool next_live = walk.live;
      entry();
      auto fetch = [&](int k) {
        uint32_t exist, missing;
        live[k] = next_live;
        rows.load(p, lane, items[k], exist, missing);
        next_live = walk.live;
        entry();
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k) fetch(k);
      bool run = true;
      for (uint32_t u = 0; run;) {
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
          if (!run || !live[k]) {
            run = false;
            break;
          }
          fetch((k + kAhead) % kSets);
          const uint32_t vs = u % L::kVSlots;
          if (u >= L::kVSlots) {
            const uint32_t v = u - L::kVSlots;
            if (!warp_wait<true>(bar(C::kPvDone, v % kPSlots), (v / kPSlots) & 1, abort_addr, lim)) {
              run = false;
              break;
            }
          }
          store_items<kFmt, kLat, false, true>(items[k], sbase + L::kV + vs * L::kVSlot, w, lane);
          fence_proxy_async_cta();
          __syncwarp();
          if (lane == 0) tell_leader(C::kVFull, vs);
          ++u;
        }
      }
    }
  } else {
    more_registers<kSoftRegs>();
    if (scoring) {
      // ------------------------------------------------ Q, softmax (thread = row)
      // The two groups of four warps take the pieces in turn. A row's reference goes
      // from piece to piece through shared memory; each group has a sum of its own.
      const uint32_t group = warp >> 2, quad = warp & 3;
      const uint32_t t = tid & 127;
      const uint32_t lane_base = (32 * quad) << 16;
      const int row = 128 * static_cast<int>(part) + static_cast<int>(t);  // of the row tile
      const uint32_t out_rank = kPair + part;
      const float c = p.score_scale;
      const uint64_t c2 = f32x2(c, c);
      uint32_t i0 = 0, u0 = 0, joined = 0;  // tiles, pieces and results of two groups before
      bool ok = true;
      Pieces<kPair> pieces(p, cluster);
      for (uint32_t item = 0; ok && pieces.next(); ++item) {
        const uint32_t n = static_cast<uint32_t>(pieces.end - pieces.begin) * kPair;
        // the MMAs that read the Q before are done
        if (i0 > 0) ok = warp_wait(bar(C::kSFull, (i0 - 1) % L::kSBufs), ((i0 - 1) / L::kSBufs) & 1, abort_addr, lim);
        if (!ok) break;
        tc_fence_after();
        {  // each group writes half of Q
          const bool mine = row < pieces.rows;
          const uint4* ql = reinterpret_cast<const uint4*>(p.q_lat + (pieces.row0 + row) * kLatent) + 32 * group;
          const uint4* qr = reinterpret_cast<const uint4*>(p.q_rope + (pieces.row0 + row) * kRope) + 4 * group;
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            uint4 v[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) v[y] = mine ? __ldg(ql + 8 * x + y) : z;
            uint32_t h[32];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const uint4 f = to_f16x8(v[y], p.lat_mult);
              h[4 * y] = f.x, h[4 * y + 1] = f.y, h[4 * y + 2] = f.z, h[4 * y + 3] = f.w;
            }
            tmem_st32(tmem + lane_base + 128u * group + 32u * x, h);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint4 f = to_f16x8(mine ? __ldg(qr + y) : z, p.rope_mult);
            st_shared_v4(sbase + L::kQRope + swizzled(t, 4 * group + y), f.x, f.y, f.z, f.w);
          }
          tmem_st_wait();
          tc_fence_before();
          fence_proxy_async_cta();
          __syncwarp();
          if (lane == 0) tell_leader(C::kQFull, 0);
        }
        // keys that the row sees
        const int32_t sees = pieces.base + 1 +
                             static_cast<int32_t>((pieces.row0 - pieces.first_row + min(row, pieces.rows - 1)) /
                                                  p.num_heads);
        float m = -INFINITY, l = 0.f;  // the reference that l is relative to
        for (uint32_t x = (u0 ^ group) & 1; x < n; x += 2) {
          const uint32_t u = u0 + x, ps = u % kPSlots, i = i0 + x / kPair, h = x % kPair, b = i % L::kSBufs;
          ok = warp_wait(bar(C::kSFull, b), (i / L::kSBufs) & 1, abort_addr, lim);
          if (!ok) break;
          tc_fence_after();
          uint32_t s[2][32];
          const uint32_t s_addr = tmem + lane_base + L::kSCol + kTileKeys * b + kPieceKeys * h;
          tmem_ld32(s_addr, s[0]);
          tmem_ld32(s_addr + 32u, s[1]);
          // keys of the piece that the row could see, and (lane j) of keys 8 j .. 8 j + 7 those that exist
          const int32_t room = sees - ((pieces.begin + static_cast<int32_t>(x / kPair)) * kTileKeys +
                                       kPieceKeys * static_cast<int32_t>(h));
          uint32_t exist = 0xffu;
          if (lane < 8) {
            const uint32_t v =
                ld_shared_u32(ctl + C::kMissing + C::kMissingBytes * (i % C::kMissingTiles) + 32 * h + 4 * lane);
            if ((v >> 8) == ((i + 1) & 0xffffffu)) exist = v & 0xffu;
          }
          const bool all = __all_sync(0xffffffffu, room >= kPieceKeys && exist == 0xffu);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) tell_leader(C::kSEmpty, b);  // S is read
          uint32_t bits[2] = {0xffffffffu, 0xffffffffu};  // the keys that the row sees
          if (!all) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              uint32_t word = 0;
#pragma unroll
              for (int y = 0; y < 4; ++y) word |= __shfl_sync(0xffffffffu, exist, 4 * a + y) << (8 * y);
              const int32_t seen = room - 32 * a;
              bits[a] = seen >= 32 ? word : seen <= 0 ? 0u : word & ((1u << seen) - 1u);
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
            ok = warp_wait(bar(C::kRefDone, 4 * (v & 1) + quad), (v >> 1) & 1, abort_addr, lim);
            if (!ok) break;
          }
          const float before =
              x > 0 ? __uint_as_float(ld_shared_u32(sbase + L::kRef + 512 * ((u - 1) & 1) + 4 * t)) : -INFINITY;
          const bool moves = top > before + kTau;  // also the first score that the row sees
          const float ref = moves ? top - kHeadroom : before;
          st_shared_u32(sbase + L::kRef + 512 * (u & 1) + 4 * t, __float_as_uint(ref));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kRefDone, 4 * (u & 1) + quad));
          if (ref != m) {
            l *= m == -INFINITY ? 0.f : ex2(m - ref);
            m = ref;
          }
          const float nm = m == -INFINITY ? 0.f : -m;
          const uint64_t nm2 = f32x2(nm, nm);
          if (u >= kPSlots)
            ok = warp_wait<true>(bar(C::kPvDone, ps), ((u / kPSlots) & 1) ^ 1, abort_addr, lim);
          if (!ok) break;
          const uint32_t dst = sbase + L::kStaged + ps * kPBytes;
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t pk[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int at = 8 * q + 2 * y;
                float e0, e1;
                split_f32x2(fma_f32x2(f32x2(__uint_as_float(s[a][at]), __uint_as_float(s[a][at + 1])), c2, nm2),
                            e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                if (!all) {
                  if (!((bits[a] >> at) & 1u)) e0 = 0.f;
                  if (!((bits[a] >> (at + 1)) & 1u)) e1 = 0.f;
                }
                sum[y & 1] = add_f32x2(sum[y & 1], f32x2(e0, e1));
                pk[y] = pack_f16x2(e0, e1);
              }
              st_shared_v4(dst + swizzled(t, 4 * a + q), pk[0], pk[1], pk[2], pk[3]);
            }
          {
            float e0, e1;
            split_f32x2(add_f32x2(sum[0], sum[1]), e0, e1);
            l += e0 + e1;
          }
          if (x + 2 == n) {  // the other group ends the result
            st_shared_u32(sbase + L::kSums + 512 * (joined & 1) + 4 * t, __float_as_uint(l));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kSumDone, 4 * (joined & 1) + quad));
          }
          // What goes with the piece, rarely: factors, and behind the last one what the
          // output is to be multiplied by
          const bool last = x + 1 == n;
          const bool rescale = __any_sync(0xffffffffu, moves && before != -INFINITY);
          if (rescale || last) {
            if (rescale) {
              const float alpha = !moves ? 1.f : before == -INFINITY ? 0.f : ex2(before - ref);
              st_cluster_u32(map_rank(sbase + L::kFactor + 512 * ps + 4 * t, out_rank), __float_as_uint(alpha));
              if (lane == 0) st_cluster_u32(map_rank(sbase + L::kTag + 16 * ps + 4 * quad, out_rank), u + 1);
            }
            if (last) {
              if (n > 1) {
                ok = warp_wait(bar(C::kSumDone, 4 * (joined & 1) + quad), (joined >> 1) & 1, abort_addr, lim);
                if (!ok) break;
                const float other = __uint_as_float(ld_shared_u32(sbase + L::kSums + 512 * (joined & 1) + 4 * t));
                l += before == -INFINITY ? 0.f : other * ex2(before - ref);
              }
              st_cluster_u32(map_rank(sbase + L::kFinal + 512 * (item % L::kFinals) + 4 * t, out_rank),
                             __float_as_uint(l == 0.f ? 0.f : p.out_mult / l));
            }
            if (lane == 0) st_shared_u32(ctl + C::kNoted + 4 * ps, u + 1);
          }
          fence_proxy_async_cta();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kStaged, ps));
          if (last && row < pieces.rows) {
            const float lse = l == 0.f ? -INFINITY : (m + lg2(l)) * kLn2;
            if (!pieces.whole) p.part_lse[static_cast<int64_t>(pieces.slot) * (128 * kPair) + row] = lse;
            else if (p.lse != nullptr) p.lse[pieces.row0 + row] = lse;
          }
        }
        if (n > 1) ++joined;
        i0 += n / kPair;
        u0 += n;
      }
    } else {
      // ------------------------------------------------ rescaling and output (thread = row)
      // Each group of four warps has half of the columns.
      const uint32_t group = warp >> 2, quad = warp & 3, t = tid & 127;
      const uint32_t o_addr = tmem + ((32 * quad) << 16) + 256u * group;
      const int row = 128 * static_cast<int>(part) + static_cast<int>(t);
      uint32_t tasks = 0;
      bool ok = true;
      Pieces<kPair> pieces(p, cluster);
      for (uint32_t item = 0; ok && pieces.next(); ++item) {
        for (bool rescaling = true; rescaling;) {
          ok = warp_wait(bar(C::kTask, 0), tasks & 1, abort_addr, lim);
          if (!ok) break;
          ++tasks;
          const uint32_t word = ld_shared_u32(ctl + C::kTaskWord);
          const uint32_t u = word >> 1, ps = u % kPSlots;
          rescaling = (word & 1u) == 0u;
          if (rescaling) {
            if (ld_shared_u32(sbase + L::kTag + 16 * ps + 4 * quad) == u + 1) {
              // after a piece of the same rows, whose MMAs (and all before) have to be done
              ok = warp_wait<true>(bar(C::kPvDone, (u - 1) % kPSlots), ((u - 1) / kPSlots) & 1, abort_addr, lim);
              if (!ok) break;
              tc_fence_after();
              const float alpha = __uint_as_float(ld_shared_u32(sbase + L::kFactor + 512 * ps + 4 * t));
#pragma unroll 1
              for (int y = 0; y < 8; ++y) {
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
            ok = warp_wait<true>(bar(C::kPvDone, ps), (u / kPSlots) & 1, abort_addr, lim);
            if (!ok) break;
            tc_fence_after();
            const float fin = __uint_as_float(ld_shared_u32(sbase + L::kFinal + 512 * (item % L::kFinals) + 4 * t));
            const bool mine = row < pieces.rows;
            const bool f32 = !pieces.whole || p.out_fp32;
            float* wide = pieces.whole
                              ? static_cast<float*>(p.out) + (pieces.row0 + row) * kLatent
                              : p.part_out + (static_cast<int64_t>(pieces.slot) * (128 * kPair) + row) * kLatent;
            wide += 256 * group;
            uint16_t* narrow = static_cast<uint16_t*>(p.out) + (pieces.row0 + row) * kLatent + 256 * group;
#pragma unroll 1
            for (int y = 0; y < 8; ++y) {
              uint32_t r[32];
              tmem_ld32(o_addr + 32u * y, r);
              tmem_ld_wait();
              float v[32];
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(r[q]) * fin;
              if (!mine) continue;
              if (f32) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  *reinterpret_cast<float4*>(wide + 32 * y + 4 * q) =
                      make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
              } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  *reinterpret_cast<uint4*>(narrow + 32 * y + 8 * q) =
                      make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                 pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
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
    const uint32_t scored = ld_shared_u32(ctl + C::kScored), summed = ld_shared_u32(ctl + C::kSummed);
    const uint32_t sent = ld_shared_u32(ctl + C::kSent);
    if (scored > 0) drain(bar(C::kSFull, (scored - 1) % L::kSBufs), ((scored - 1) / L::kSBufs) & 1);
    if (sent > 0) drain(bar(C::kPFull, (sent - 1) % kPSlots), ((sent - 1) / kPSlots) & 1);
    if (summed > 0) drain(bar(C::kPvDone, (summed - 1) % kPSlots), ((summed - 1) / kPSlots) & 1);
  }
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    free_tmem<kPair>(tmem);
  }
  cluster_sync();
}

// ------------------------------------------------------------------ merging
// Row tiles that several clusters worked on: out = sum_p w_p out_p / sum_p w_p
// with w_p = exp(lse_p - max). A warp has a row; the border between two
// clusters' shares that is the first inside a row tile stands for it.
template <int kPair>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p) {
  constexpr int kRows = 128 * kPair;
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
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
  for (int64_t x = me; x < static_cast<int64_t>(p.clusters - 1) * kRows; x += warps) {
    const int c = 1 + static_cast<int>(x / kRows), row = static_cast<int>(x % kRows);
    const int64_t at = c * share;
    if (at >= units) break;
    const int t = __ldcg(p.first + c);  // whose units reach to c's first one, or begin there
    // first[c] is the last row tile that begins at or before `at`
    const RowTile tile = p.tiles[t];
    const int64_t a = tile.unit, b = p.tiles[t + 1].unit;
    if (a == at || a < at - share) continue;  // not cut here, or before
    int32_t start, len;
    const int64_t n = static_cast<int64_t>(new_tokens(p, tile.seq, start, len)) * p.num_heads;
    const int64_t first_row = static_cast<int64_t>(tile.index) * kRows;
    if (row >= n - first_row) continue;
    const int64_t k0 = a + kTileOverhead<kPair>;
    const int c1 = static_cast<int>((b - 1) / share);
    // the parts: cluster c - 1 to c1, those that have key tiles
    auto has = [&](int q) {
      const int64_t lo = max(q * share - k0, int64_t{0}), hi = min((q + 1) * share, b) - k0;
      return hi > lo;
    };
    auto lse_at = [&](int q) {
      return p.part_lse + static_cast<int64_t>(2 * q + (a >= q * share ? 1 : 0)) * kRows + row;
    };
    int q0 = c - 1;
    while (q0 < c1 && !has(q0)) ++q0;
    if (q0 == c1) continue;  // all key tiles in one cluster: it wrote the result
    float top = -INFINITY;
    bool nan = false;
    for (int q = q0; q <= c1; ++q) {
      const float z = __ldcg(lse_at(q));
      nan |= z != z;
      top = fmaxf(top, z);
    }
    float acc[16] = {};
    float tot = 0.f;
    if (top != -INFINITY) {
      for (int q = q0; q <= c1; ++q) {
        const float w = ex2((__ldcg(lse_at(q)) - top) * kLog2e);
        tot += w;
        if (w == 0.f) continue;
        const float* from =
            p.part_out + (static_cast<int64_t>(2 * q + (a >= q * share ? 1 : 0)) * kRows + row) * kLatent;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(from + 128 * y + 4 * lane));
          acc[4 * y] += w * v.x;
          acc[4 * y + 1] += w * v.y;
          acc[4 * y + 2] += w * v.z;
          acc[4 * y + 3] += w * v.w;
        }
      }
    }
    const float inv = nan ? NAN : tot > 0.f ? 1.f / tot : 0.f;
    const int64_t to = static_cast<int64_t>(start) * p.num_heads + first_row + row;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const float v0 = acc[4 * y] * inv, v1 = acc[4 * y + 1] * inv, v2 = acc[4 * y + 2] * inv,
                  v3 = acc[4 * y + 3] * inv;
      if (p.out_fp32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to * kLatent + 128 * y + 4 * lane) =
            make_float4(v0, v1, v2, v3);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to * kLatent + 128 * y + 4 * lane) =
            make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3));
    }
    if (lane == 0 && p.lse != nullptr)
      p.lse[to] = nan ? NAN : tot > 0.f ? top + lg2(tot) * kLn2 : -INFINITY;
  }
}

// ------------------------------------------------------------------ host
// Two SMs a sequence's rows where they fill more than one and a half times 128.
int pair_of(int32_t num_q, int32_t num_heads, int32_t num_seqs) {
  return 2 * static_cast<int64_t>(num_q) * num_heads > 3 * int64_t{128} * num_seqs ? 2 : 1;
}

struct ChunkSpace {
  size_t tiles, first, failed, lse, out, bytes;  // offsets
  int32_t max_tiles;
};
ChunkSpace chunk_space(int32_t num_q, int32_t num_heads, int32_t num_seqs) {
  const int pair = pair_of(num_q, num_heads, num_seqs);
  const int64_t rows = 128 * pair;
  ChunkSpace s;
  const int64_t tiles = static_cast<int64_t>(num_q) * num_heads / rows + (num_seqs < num_q ? num_seqs : num_q);
  s.max_tiles = static_cast<int32_t>(tiles);
  s.tiles = 64;
  s.first = s.tiles + sizeof(RowTile) * static_cast<size_t>(tiles + 1);
  s.failed = s.first + 4 * kMaxClusters;
  s.lse = s.failed + 4 * kMaxClusters;
  s.out = s.lse + 4 * 2 * kMaxClusters * 128;
  s.bytes = s.out + size_t{4} * 2 * kMaxClusters * 128 * kLatent;
  return s;
}
static_assert(sizeof(RowTile) == 16 && sizeof(Plan) <= 64 && (4 * kMaxClusters) % 16 == 0, "workspace");

bool chunk_shape_ok(int32_t num_q, int32_t num_heads, int32_t num_seqs) {
  return num_q >= 0 && num_heads >= 1 && num_heads <= NVFP4_MLA_MAX_HEADS && num_seqs >= 1 &&
         num_seqs <= NVFP4_MLA_MAX_PLAN_SEQS &&
         static_cast<int64_t>(num_q) * num_heads <= INT32_MAX;
}

// Clusters of a kernel that the device holds at once, asked once a device.
template <int kFmt, int kPair, bool kRuns>
int32_t resident_clusters(int device, cudaLaunchConfig_t cfg, int sms, int* clusters) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int n = device < kDevices ? known[device].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(sms / (2 * kPair) * (2 * kPair)));
    if (cudaOccupancyMaxActiveClusters(&n, chunk_kernel<kFmt, kPair, kRuns>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return NVFP4_MLA_ERR_LAUNCH;
    }
    n = n < kMaxClusters / kPair ? n : kMaxClusters / kPair;
    if (device < kDevices) known[device].store(n, std::memory_order_relaxed);
  }
  *clusters = n;
  return NVFP4_MLA_OK;
}

template <int kFmt, int kPair, bool kRuns>
int32_t launch_chunk(ChunkParams p, int device, int sms, cudaStream_t stream) {
  constexpr size_t smem = ChunkLayout<kPair>::kBytes;
  const size_t plan_smem = 4 * static_cast<size_t>(p.num_seqs);
  // limits of the process: the same in every call
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(chunk_kernel<kFmt, kPair, kRuns>),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
      (plan_smem > 40 * 1024 &&
       cudaFuncSetAttribute(reinterpret_cast<const void*>(chunk_plan_kernel<kPair>),
                            cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * NVFP4_MLA_MAX_PLAN_SEQS) != cudaSuccess)) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kChunkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * kPair;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (int32_t st = resident_clusters<kFmt, kPair, kRuns>(device, cfg, sms, &p.clusters)) return st;
  if (p.invalid_count != nullptr) {
    chunk_check_kernel<<<p.num_seqs < 4 * sms ? p.num_seqs : 4 * sms, 256, 0, stream>>>(p);
    if (int32_t st = launch_status()) return st;
  }
  chunk_plan_kernel<kPair><<<1, kPlanThreads, plan_smem, stream>>>(p);
  if (int32_t st = launch_status()) return st;
  cfg.gridDim = dim3(static_cast<unsigned>(p.clusters * 2 * kPair));
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, chunk_kernel<kFmt, kPair, kRuns>, p) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  cudaLaunchConfig_t last = {};
  last.gridDim = dim3(static_cast<unsigned>(4 * sms));
  last.blockDim = dim3(256);
  last.stream = stream;
  last.attrs = attr + 1;
  last.numAttrs = 1;
  if (cudaLaunchKernelEx(&last, chunk_merge_kernel<kPair>, p) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  return NVFP4_MLA_OK;
}

template <int kFmt, int kPair>
int32_t launch_pages(const ChunkParams& p, bool runs, int device, int sms, cudaStream_t stream) {
  return runs ? launch_chunk<kFmt, kPair, true>(p, device, sms, stream)
              : launch_chunk<kFmt, kPair, false>(p, device, sms, stream);
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
  p.score_scale = fabsf(sm_scale) * lat * kLog2e;
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
  const int pair = pair_of(num_q, num_heads, num_seqs);
  const bool runs = page_size % kPieceKeys == 0;
  if (fp8)
    return pair == 2 ? launch_pages<NVFP4_MLA_ROW_FP8_576, 2>(p, runs, dev, sms, s)
                     : launch_pages<NVFP4_MLA_ROW_FP8_576, 1>(p, runs, dev, sms, s);
  return pair == 2 ? launch_pages<NVFP4_MLA_ROW_NVFP4_352, 2>(p, runs, dev, sms, s)
                   : launch_pages<NVFP4_MLA_ROW_NVFP4_352, 1>(p, runs, dev, sms, s);
}
