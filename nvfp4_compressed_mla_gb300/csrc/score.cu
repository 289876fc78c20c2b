// score.cu -- index scores of every visible position of every query token, on
// the block-scaled FP4 tensor cores (tcgen05 kind::mxf4nvf4).
//
// Keys and queries are stored as the tensor cores take them (E2M1 codes, one
// E4M3 scale per 16 values along the contraction), so nothing is dequantised:
// per tile of 128 positions and query token, D = K Q^T (M = 128 positions,
// N = heads, K = 128 in two steps), and the epilogue adds up
// sum_j w_j max(0, D_j) in fp32, thread = position.
//
// The bound is HBM for one query token per sequence: 72 bytes a position
// against 2 * 128 * heads FP4 flop. With several query tokens a sequence, a
// tile is read once for up to `group` of them and the epilogue's fp32 work
// (one max and one fma per position and head) bounds it.
//
// One persistent CTA per SM. All visible (tile, query token run) pairs form
// one list, and each CTA takes a contiguous part of it of equal cost, so one
// long sequence fills the device as well as many short ones. Runs are
// consecutive query tokens of one sequence, at most `group` of them.
//
// Positions go through in steps of 256: each role is one or a few warps whose
// handshakes and address arithmetic cost hundreds of cycles a step, however
// large the step is. Two neighbouring rows of a page are one 128-byte line in
// shared memory, as tensor copies take time per line: the MMA's row R holds
// position 2 R in the line's first 64 bytes and 2 R + 1 in the others, and a
// step's two tiles are its even and its odd positions.
//
//   warps 0-11   epilogue: three sets of four; a set takes every third
//                (step, query token) unit, warp w the rows 32 (w % 4).. of both
//                tiles (more than 64 heads: two sets, one tile after the other)
//   warps 12, 13 copy the codes of every other step: resolve the pages through
//                the block table (two turns ahead), one tensor copy per page,
//                swizzled on the way; all stages in flight
//   warps 14-17  take turns in loading a step's scales (one turn ahead) and
//                laying them out in tensor memory
//   (page sizes that are no power of two or below 16: warps 12-15 copy row by row
//   with cp.async instead)
//   warps 18, 19 issue the MMAs of every other step (more than 64 heads: warp 18
//                alone); warp 18 copies the next run's queries meanwhile
//
// A first kernel encodes the queries, once for all CTAs that score a run, into
// images of what the MMAs and the epilogue read of them.
//
// Every wait is bounded; when one runs out the CTA's roles unwind, what is in
// flight is drained, and the CTA's status word says so.
//
// Measured (GB300, device time, 64 heads): 66 sequences of about 146000 tokens,
// one query token each, 127 us: 694 MB of keys and 36 MB of scores at 5.7 TB/s,
// 0.84 of a copy's rate (217 us with the copies row by row). Per step of 256
// positions an SM takes about 1000 cycles, 790 of which the copy rate explains.
// 32 sequences x 15 query tokens x 65536 positions 325 us (1590 TFLOP/s of FP4
// products), two thirds of the issue slots taken by the sums over the heads; one
// sequence of a million tokens 23 us (72 MB, the kernel's start included); one
// of 4096 tokens, 16 heads 7.7 us.
#include <math.h>
#include <string.h>

#include "select_common.cuh"
#include "tc_ptx.cuh"

namespace nvfp4_mla {
namespace {

constexpr int kScoreThreads = 640;
constexpr int kEpiWarps = 12;
constexpr int kLoadWarp0 = 12, kLoadWarps = 4;
constexpr int kCopyWarps = 2, kScaleWarp0 = 14, kScaleWarps = 4;  // with tensor copies
constexpr int kMmaWarp0 = 18;
constexpr int kMaxStages = 7;     // steps in shared memory
// Resolved-position masks of the last tiles; more than there can be between a
// step's scales and its epilogue (the stages and the accumulator slots).
constexpr int kMaskRing = 32;
// Query tokens of a run: 512 query tokens a sequence, 32 heads, 16384 positions
// 262 us with 4, 281 with 2, 353 with 1. More would take shared memory from the
// stages.
constexpr int kMaxGroup = 4;
constexpr int kStep = 256;                             // positions
constexpr int kStepTiles = kStep / kScoreTile;         // 2
constexpr int kStepCodes = kStep * kIndexCodes;        // 128 lines of 128 bytes, 128-byte swizzle
constexpr int kTileScales = 1024;                      // two K halves of 128 x 4 scale bytes
constexpr int kStageBytes = kStepCodes + kStepTiles * kTileScales;
constexpr int kMaskBytes = kMaskRing * 4 * 4;
// A run's cost per step: its query tokens' epilogues and the step's load. 32
// sequences x 15 query tokens, 64 heads, 65536 positions: 325 us with 4 to 1,
// 338 without the load, 334 with 1 to 1, 342 with 1 to 2, 352 with 1 to 4; runs
// of one length are cut the same by all of them.
constexpr int kTokenCost = 4, kLoadCost = 1;
// Tensor memory columns: accumulator slots, then scales of Q (eight per query
// token of a run, a set for each MMA warp), then of K (eight per tile of a
// stage).
constexpr uint32_t kSfbCol = 384;
// Stages of a run's length: what tensor memory holds scales for. A stage's
// round (copies under way, MMAs, release) takes several thousand cycles, so
// the copies in flight set the rate.
__host__ __device__ constexpr int mma_warps(int chunks) { return chunks <= 2 ? 2 : 1; }
__host__ __device__ constexpr int stage_count(int chunks, int group) {
  const int n = (static_cast<int>(kTmemCols - kSfbCol) / 8 - mma_warps(chunks) * group) / kStepTiles;
  return n < kMaxStages ? n : kMaxStages;
}

// Instruction descriptor, kind::mxf4nvf4: E2M1 A (bit 7) and B (bit 10), both
// K-major, E4M3 scales, N >> 3 at 17, M >> 4 at 24, K = 64.
__host__ __device__ constexpr uint32_t score_idesc(int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}
// For `chunks` of 32 heads: tiles of an accumulator slot, slots, and sets of
// epilogue warps. A set waits for a slot's phase by its parity, so it must not
// come to a slot before the slot's last content is there: a slot is one set's
// (64 heads or fewer), or units complete in order and, with s sets, the
// contents of the s - 1 units between two of its own fit into the slots.
__host__ __device__ constexpr int slot_tiles(int chunks) { return chunks <= 2 ? 2 : 1; }
__host__ __device__ constexpr int acc_slots(int chunks) {
  return 384 / (32 * chunks * slot_tiles(chunks));
}
__host__ __device__ constexpr int epi_sets(int chunks) { return chunks <= 2 ? 3 : 2; }

// K-major operand with 64-byte rows in 64-byte swizzle: 8-row groups of 512 bytes.
__device__ __forceinline__ uint64_t sw64_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(4) << 61);
}
// The same with 128-byte rows in 128-byte swizzle: 8-row groups of 1024 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
// 16-byte chunk (0..3) of position x of a step.
__device__ __forceinline__ uint32_t code_off(uint32_t x, uint32_t chunk) {
  const uint32_t line = x >> 1;
  return line * 128u + ((((x & 1u) * 4u + chunk) ^ (line & 7u)) << 4);
}
__device__ __forceinline__ uint32_t sw64_off(uint32_t row, uint32_t chunk) {
  return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}
// 32 rows of 16 bytes without swizzle: 8-row groups of 128 bytes.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
// Scale byte g (0..7) of row r (0..127): per K half, row r % 32 holds the four
// bytes of rows r, r + 32, .. in turn.
__device__ __forceinline__ uint32_t scale_off(uint32_t r, uint32_t g) {
  return (g >> 2) * 512u + (r & 31u) * 16u + (r >> 5) * 4u + (g & 3u);
}
// 512 bytes of scales -> four columns of tensor memory, in all lane quadrants
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 16 or 4 bytes, or zeros where `live` is false
__device__ __forceinline__ void cp_async16_z(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16u : 0u)
               : "memory");
}
__device__ __forceinline__ void cp_async4_z(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 4u : 0u)
               : "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
// 8 consecutive TMEM columns of this thread's lane
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// 2 max(0, x), exact, NaN stays NaN: an addition; the maximum takes the slower
// integer pipe.
__device__ __forceinline__ float twice_relu(float x) { return x + fabsf(x); }
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  return lo + hi;
}
// True in one lane of the warp, the same one every time; the compiler knows
// that it is one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// One warp's bounded wait: it leaves together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort_addr,
                                          long long limit) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_addr, limit)) != 0;
}

// Bounded wait at the end, whether the CTA aborts or not.
__device__ __noinline__ void drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_test(bar, parity) && clock64() - t0 < (1ll << 31)) {
  }
}

struct Bars {  // byte offsets in the control block
  static constexpr int kFull = 0, kEmpty = kFull + 8 * kMaxStages,
                       kDFull = kEmpty + 8 * kMaxStages,
                       kDEmpty = kDFull + 64, kQFull = kDEmpty + 64, kQEmpty = kQFull + 16,
                       kDrain = kQEmpty + 16, kTurn = kDrain + 16, kScaleDrain = kTurn + 16,
                       kTmem = kScaleDrain + 8 * kScaleWarps, kAbort = kTmem + 4,
                       kStart = kAbort + 4,
                       // steps that each copying warp has issued, and each scale
                       // warp committed, when it ends
                       kIssued = kStart + 32, kCommitted = kIssued + 4 * kCopyWarps,
                       kEnd = kCommitted + 4 * kScaleWarps;
};
static_assert(Bars::kStart % 8 == 0, "start words");
// An aborted CTA's code copies land before it ends. Every role has ended: no
// one else arrives at the stages any more, except for scale commits under way,
// which are counted. Step n is copy warp n % kCopyWarps' and scale warp
// n % kScaleWarps'. A stage is issued once its last content has been used, so
// only the newest `stages` steps can be in flight; a stage that is copied and
// has no scales lacks exactly the scale warp's arrival.
__device__ __noinline__ void drain_codes(uint32_t ctl, uint32_t stages) {
  uint32_t end = 0;  // behind the newest step that was issued
  for (uint32_t w = 0; w < kCopyWarps; ++w) {
    const uint32_t n = ld_shared_u32(ctl + Bars::kIssued + 4 * w);
    if (n > 0) end = max(end, w + (n - 1) * kCopyWarps + 1);
  }
  for (uint32_t n = end > stages ? end - stages : 0; n < end; ++n) {
    if (n / kCopyWarps >= ld_shared_u32(ctl + Bars::kIssued + 4 * (n % kCopyWarps))) continue;
    const uint32_t full = ctl + Bars::kFull + 8 * (n % stages);
    if (n / kScaleWarps >= ld_shared_u32(ctl + Bars::kCommitted + 4 * (n % kScaleWarps)))
      mbar_arrive(full);
    drain(full, (n / stages) & 1u);
  }
}
constexpr int kCtl = kMaskBytes;  // the control block follows the masks
constexpr int kStageBase = (kCtl + Bars::kEnd + 1023) / 1024 * 1024;  // stages, then two Q buffers

constexpr int kImageLine = 512;  // images as lines, for tensor copies
// A query token's image: codes in 64-byte swizzle, scales, weights (zeros past
// num_heads), whole swizzle atoms.
__host__ __device__ constexpr int image_scales(int heads_pad) { return heads_pad * kIndexCodes; }
__host__ __device__ constexpr int image_weights(int heads_pad) {
  return image_scales(heads_pad) + kTileScales;
}
__host__ __device__ constexpr int image_bytes(int heads_pad) {
  return (image_weights(heads_pad) + heads_pad * 4 + kImageLine - 1) / kImageLine * kImageLine;
}

// One thread per group of 16 values; a CTA per query token.
__global__ void __launch_bounds__(NVFP4_MLA_MAX_HEADS* kIndexScales)
    encode_kernel(const uint8_t* __restrict__ q_index, const float* __restrict__ weights,
                  int32_t num_heads, int32_t heads_pad, uint8_t* __restrict__ images) {
  cudaTriggerProgrammaticLaunchCompletion();
  const int64_t t = blockIdx.x;
  const int g = threadIdx.x % kIndexScales, h = threadIdx.x / kIndexScales;
  uint32_t lo = 0, hi = 0, sc = 0;
  float weight = 0.f;
  if (h < num_heads) {
    const int64_t head = t * num_heads + h;
    const uint8_t* src = q_index + head * (kIndexDim * 2) + g * (2 * kGroup);
    const uint4 a = ld_nc_v4(src), b = ld_nc_v4(src + 16);
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float s;
    sc = quantize_group(v, lo, hi, s);
    if (g == 0) weight = __ldg(weights + head);
  }
  uint8_t* image = images + t * image_bytes(heads_pad);
  *reinterpret_cast<uint2*>(image + sw64_off(h, g >> 1) + (g & 1) * 8) = make_uint2(lo, hi);
  image[image_scales(heads_pad) + scale_off(h, g)] = static_cast<uint8_t>(sc);
  if (g == 0) *reinterpret_cast<float*>(image + image_weights(heads_pad) + h * 4) = weight;
}

struct ScoreParams {
  SelectParams s;
  int32_t group;
  int32_t ctas;
  int32_t stages;
  int32_t seg_rows;    // rows of a tensor copy; 0: copies row by row
  int32_t page_shift;  // log2 of the page size (tensor copies)
};

// one box of a 2-D tensor map at (x, y)
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* tm, int32_t x,
                                            int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// one box of a 3-D tensor map at (0, y, z)
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}
// Largest of the bytes (E4M3 scales, positive) of words, in the high bytes of
// 16-bit values, two of which one instruction compares.
struct TopByte {
  uint32_t even = 0, odd = 0;
  __device__ __forceinline__ void add(uint32_t v) {
    even = __vmaxu2(even, v << 8);
    odd = __vmaxu2(odd, v);
  }
  __device__ __forceinline__ uint32_t of_warp() const {  // at most 448
    const uint32_t m = __vmaxu2(even, odd);
    return min(__reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16)) >> 8, 0x7Eu);
  }
};

// A place in the ring of stages and the parity of its round.
struct Ring {
  uint32_t stage = 0, phase = 0, stages;
  __device__ __forceinline__ explicit Ring(uint32_t n) : stages(n) {}
  __device__ __forceinline__ void advance(uint32_t steps) {  // at most `stages`
    stage += steps;
    if (stage >= stages) stage -= stages, phase ^= 1u;
  }
};

// A CTA's part of the list of steps: from step start_t of the run that begins
// with query token start_q to step end_t - 1 of that which begins with end_q.
struct Part {
  int32_t start_q, start_t, end_q, end_t;
};

// The runs of query tokens whose steps a CTA scores, walked by one warp. Lane
// i holds query token i of the current run; the next run's words are loaded
// while the current one is worked on. Every role has a copy of this code, so
// it holds no division.
struct Walk {
  int32_t q, count, seq, t0, t1;  // run; steps t0 .. t1 - 1 are this CTA's
  int32_t seen;                   // lane i: positions to score of token q + i
  int32_t most;                   // the highest of them
  int32_t next_q, next_t;
  int32_t next_seq, next_pos;     // lane i: words of token next_q + i
  int32_t next_lim;               // query tokens from next_q to the end of its group
  int32_t end_q, end_t;

  __device__ __forceinline__ void load(const ScoreParams& p) {
    const int32_t lane = threadIdx.x & 31;
    next_seq = next_pos = -1;
    if (lane < next_lim) {
      next_seq = __ldg(p.s.q_seq + next_q + lane);
      next_pos = __ldg(p.s.q_pos + next_q + lane);
    }
  }
  __device__ __forceinline__ void begin(const ScoreParams& p, const Part& part) {
    next_q = part.start_q, next_t = part.start_t;
    end_q = part.end_q, end_t = part.end_t;
    next_lim = min(p.group - next_q % p.group, p.s.num_q - next_q);
    load(p);
  }
  // Moves to the next run with steps of this CTA; false when there is none.
  __device__ __forceinline__ bool next(const ScoreParams& p) {
    const int32_t lane = threadIdx.x & 31;
#pragma unroll 1
    while (next_q <= end_q && next_lim > 0) {
      q = next_q;
      seq = __shfl_sync(0xffffffffu, next_seq, 0);
      const uint32_t same = __ballot_sync(0xffffffffu, lane < next_lim && next_seq == seq);
      count = __ffs(~same) - 1;  // leading lanes; next_lim < 32
      seen = lane < count ? scored_positions(p.s, seq, next_pos) : 0;
      next_q += count, next_lim -= count;
      if (next_lim == 0) next_lim = min(p.group, p.s.num_q - next_q);
      load(p);
      most = static_cast<int32_t>(__reduce_max_sync(0xffffffffu, seen));
      t0 = next_t, next_t = 0;
      t1 = q == end_q ? end_t : (most + (kStep - 1)) / kStep;
      if (t0 < t1) return true;
    }
    return false;
  }
};

// One of `warps` warps that take turns at a CTA's steps.
struct Turns {
  int32_t step = 0, wait, stride;  // wait: steps until this warp's next
  uint32_t it = 0;                 // number of the step among the CTA's
  Ring at;
  __device__ __forceinline__ Turns(int32_t first, int32_t warps, uint32_t stages)
      : wait(first), stride(warps), at(stages) {}
  // Goes on to this warp's next step; false when there is none. Before the
  // first call walk.t1 is 0.
  __device__ __forceinline__ bool next(Walk& walk, const ScoreParams& p) {
#pragma unroll 1
    while (true) {
      const int32_t skip = min(wait, walk.t1 - step);
      step += skip, it += skip, wait -= skip;
      at.advance(skip);
      if (step < walk.t1) return true;
      if (!walk.next(p)) return false;
      step = walk.t0;
    }
  }
  __device__ __forceinline__ void done() {
    ++step, ++it, wait = stride - 1;
    at.advance(1);
  }
};

template <int kChunks>
__global__ void __launch_bounds__(kScoreThreads, 1)
    score_kernel(const __grid_constant__ ScoreParams p,
                 const __grid_constant__ CUtensorMap codes_map,
                 const __grid_constant__ CUtensorMap image_map) {
  constexpr int kHeads = 32 * kChunks;
  constexpr int kSlots = acc_slots(kChunks);
  constexpr int kSlotTiles = slot_tiles(kChunks);
  constexpr int kSets = epi_sets(kChunks);
  constexpr int kUnitSlots = kStepTiles / kSlotTiles;  // a unit is a step and a query token
  static_assert(kSlots >= (kSets - 1) * kUnitSlots + 1 && 4 * kSets <= kEpiWarps, "slots");
  constexpr uint32_t kSlotCols = kSlotTiles * kHeads;
  constexpr int kMmaWarps = mma_warps(kChunks);
  // with two issuing threads, whose MMAs need not complete in order
  static_assert(kMmaWarps == 1 || kSlots % kSets == 0, "slots of one set each");
  constexpr uint32_t kImage = image_bytes(kHeads);
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const uint32_t stage0 = base + kStageBase;
  const uint32_t ctl = base + kCtl;
  const uint32_t abort_addr = ctl + Bars::kAbort;
  auto bar = [ctl](int kind, int i) { return ctl + static_cast<uint32_t>(kind + 8 * i); };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long lim = p.s.wait_cycles;
  // ---- this CTA's part of the list
  __shared__ int64_t warp_cost[kScoreThreads / 32];
  const int32_t groups = (p.s.num_q + p.group - 1) / p.group;
  const int32_t per = (groups + kScoreThreads - 1) / kScoreThreads;
  const int32_t g_from = min(tid * per, groups), g_to = min(g_from + per, groups);
  auto runs = [&](auto&& each) {  // the runs of this thread's groups, in order
#pragma unroll 1
    for (int32_t q = g_from * p.group; q < min(g_to * p.group, p.s.num_q);) {
      const int32_t stop = min((q / p.group + 1) * p.group, p.s.num_q);
      const int32_t seq = __ldg(p.s.q_seq + q);
      int32_t most = 0, n = 0;
      do {
        most = max(most, scored_positions(p.s, seq, __ldg(p.s.q_pos + q + n)));
        ++n;
      } while (q + n < stop && __ldg(p.s.q_seq + q + n) == seq);
      const int32_t cost = kTokenCost * n + kLoadCost;
      each(q, static_cast<int64_t>((most + kStep - 1) / kStep) * cost, cost);
      q += n;
    }
  };
  int64_t mine = 0;
  runs([&](int32_t, int64_t cost, int32_t) { mine += cost; });
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) warp_cost[warp] = upto;
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(bar(Bars::kFull, i), p.seg_rows > 0 ? 2 : kLoadWarps);
      mbar_init(bar(Bars::kEmpty, i), 1);
    }
#pragma unroll 1
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(Bars::kDFull, i), 1);
      mbar_init(bar(Bars::kDEmpty, i), 4);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Bars::kQFull, i), 1);
      mbar_init(bar(Bars::kQEmpty, i), kEpiWarps + kMmaWarps);
    }
    for (int i = 0; i < kMmaWarps; ++i) {
      mbar_init(bar(Bars::kDrain, i), 1);
      mbar_init(bar(Bars::kTurn, i), 1);
    }
#pragma unroll 1
    for (int i = 0; i < kScaleWarps; ++i) mbar_init(bar(Bars::kScaleDrain, i), 1);
    st_shared_u32(abort_addr, 0);
    // no end inside the list: the last CTA's
    reinterpret_cast<Part*>(smem + kCtl + Bars::kStart)->end_q = INT32_MAX;
    fence_mbar_init();
  }
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kScoreThreads / 32; ++w) {
    if (w < warp) before += warp_cost[w];
    total += warp_cost[w];
  }
  const int64_t begin = total * blockIdx.x / p.ctas, end = total * (blockIdx.x + 1) / p.ctas;
  if (begin == end) {
    cudaGridDependencySynchronize();  // this grid does not end before the encoding
    if (tid == 0) p.s.status[blockIdx.x] = 0;
    return;
  }
  Part* part = reinterpret_cast<Part*>(smem + kCtl + Bars::kStart);
  before += upto - mine;
  if ((before <= begin && begin < before + mine) || (before <= end && end < before + mine)) {
    int64_t at = before;
    runs([&](int32_t q, int64_t cost, int32_t w) {
      // a step belongs to the CTA in whose share of the cost it starts
      if (at <= begin && begin < at + cost)
        part->start_q = q, part->start_t = static_cast<int32_t>((begin - at + w - 1) / w);
      if (at <= end && end < at + cost)
        part->end_q = q, part->end_t = static_cast<int32_t>((end - at + w - 1) / w);
      at += cost;
    });
  }
  if (warp == kMmaWarp0) tmem_alloc(ctl + Bars::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(ctl + Bars::kTmem);
  Walk walk;
  walk.begin(p, *part);

  // The queries are encoded; the selection may take the SMs that fall idle (it
  // waits for this grid).
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();

  const uint32_t q_base = stage0 + p.stages * kStageBytes;
  const uint32_t sfa_col = kSfbCol + 8 * kMmaWarps * p.group;
  auto q_image = [&](int buf) { return q_base + static_cast<uint32_t>(buf * p.group) * kImage; };

  if (warp < kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const uint32_t set = warp >> 2, quad = warp & 3;  // a set past kSets has no units
    const uint32_t lanes = static_cast<uint32_t>(quad) << 21;  // lane 32 * quad
    const int granule = min(p.s.block, kMaxGranule);
    const int shift = __ffs(granule) - 1;
    uint32_t first = 0, step_no = 0, run = 0;  // first: number of the step's first unit
    uint32_t done = 0;  // units of this set
    int next = set < kSets ? set : INT32_MAX;  // units from there to this set's next
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(p)) {
      const int buf = run & 1;
      ok = warp_wait(bar(Bars::kQFull, buf), (run >> 1) & 1u, abort_addr, lim);
      float* out = p.s.scores + walk.q * p.s.score_stride;
      const uint8_t* weights = smem + (q_image(buf) - base) + image_weights(kHeads);
#pragma unroll 1
      for (int32_t step = walk.t0; ok && step < walk.t1; ++step, ++step_no, first += walk.count) {
        const int32_t pos = step * kStep + 2 * (static_cast<int32_t>(quad) * 32 + lane);
        int i = next;
#pragma unroll 1
        for (; i < walk.count; i += kSets) {
          const int32_t seen = __shfl_sync(0xffffffffu, walk.seen, i);
          const auto* w = reinterpret_cast<const ulonglong2*>(weights + i * kImage);
          float score[kStepTiles];  // of positions pos, pos + 1
          uint32_t mask[kStepTiles];
#pragma unroll
          for (int u = 0; u < kUnitSlots; ++u) {
            uint32_t slot, parity;
            if constexpr (kUnitSlots == 1 && kSlots % kSets == 0) {  // every kSets-th slot is this set's
              slot = set + kSets * (done % (kSlots / kSets));
              parity = done / (kSlots / kSets) & 1u;
            } else {
              const uint32_t n = (first + i) * kUnitSlots + u;
              slot = n % kSlots;
              parity = n / kSlots & 1u;
            }
            ok = warp_wait(bar(Bars::kDFull, slot), parity, abort_addr, lim);
            if (!ok) break;
            tc_fence_after();
            if (u == 0) {
#pragma unroll
              for (int t = 0; t < kStepTiles; ++t)
                mask[t] = ld_shared_u32(base + ((step_no * kStepTiles + t) % kMaskRing * 4 + quad) * 4);
            }
            // 8 heads at a time, of all the slot's tiles: a weight's way from
            // shared memory into 32 lanes' registers costs as much as its use,
            // so each one is used for every tile. The next ones are loaded
            // while these are worked on.
            const uint32_t d = tmem + lanes + slot * kSlotCols;
            uint64_t acc[kSlotTiles][4];
#pragma unroll
            for (int t = 0; t < kSlotTiles; ++t)
              acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0;
            uint32_t v[2][kSlotTiles][8];
            ulonglong2 wj[2][2];
            auto fetch = [&](int to, int c) {
#pragma unroll
              for (int t = 0; t < kSlotTiles; ++t) tmem_ld8(d + t * kHeads + c, v[to][t]);
              wj[to][0] = w[c / 4], wj[to][1] = w[c / 4 + 1];
            };
            fetch(0, 0);
#pragma unroll 1
            for (int c = 0; c < kHeads; c += 16) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                tmem_ld_wait();
                if (h == 0) {
                  fetch(1, c + 8);
                } else if (c + 16 < kHeads) {
                  fetch(0, c + 16);
                } else {  // the slot has been read
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(bar(Bars::kDEmpty, slot));
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                  for (int t = 0; t < kSlotTiles; ++t) {
                    const uint32_t* x = v[h][t] + 4 * j;
                    fma2(acc[t][j],
                         pack2(twice_relu(__uint_as_float(x[0])), twice_relu(__uint_as_float(x[1]))),
                         wj[h][j].x);
                    fma2(acc[t][2 + j],
                         pack2(twice_relu(__uint_as_float(x[2])), twice_relu(__uint_as_float(x[3]))),
                         wj[h][j].y);
                  }
                }
              }
            }
#pragma unroll
            for (int t = 0; t < kSlotTiles; ++t)
              score[u * kSlotTiles + t] = ((sum2(acc[t][2]) + sum2(acc[t][3])) +
                                           (sum2(acc[t][0]) + sum2(acc[t][1]))) * 0.5f;
          }
          if (!ok) break;
          ++done;
#pragma unroll
          for (int t = 0; t < kStepTiles; ++t) {
            const bool real = pos + t < seen && (mask[t] >> lane & 1u) && score[t] == score[t];
            score[t] = real ? score[t] + 0.f : -INFINITY;
          }
          float* row = out + i * p.s.score_stride;
          const bool live = pos < seen;  // the row has room for both positions
          if (granule == 1) {
            if (live) *reinterpret_cast<float2*>(row + pos) = make_float2(score[0], score[1]);
          } else {
            float m = fmaxf(score[0], score[1]);
#pragma unroll
            for (int s = 1; s < kMaxGranule / 2; s <<= 1) {
              const float o = __shfl_xor_sync(0xffffffffu, m, s);
              if (s < granule / 2) m = fmaxf(m, o);
            }
            if (live && (pos & (granule - 1)) == 0) row[pos >> shift] = m;
          }
        }
        if (set < kSets) next = i - walk.count;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Bars::kQEmpty, buf));
      ++run;
    }
  } else if (p.seg_rows > 0 && warp < kLoadWarp0 + kCopyWarps) {
    // ------------------------------------------------ codes, tensor copies
    const int segs = kStep / p.seg_rows;  // lane i resolves and copies piece i of a step
    const int32_t past = static_cast<int32_t>(p.s.num_blocks);
    struct Entry {
      int32_t page, row;
      bool live;
    };
    Turns turns(warp - kLoadWarp0, kCopyWarps, p.stages);
    walk.t1 = 0;
    const bool issuer = elect_one();
    const uint32_t piece = static_cast<uint32_t>(p.seg_rows) * kIndexCodes;
    Entry e0, e1, e2;
    e0.live = e1.live = false;
    Ring at(p.stages);
    at.advance(warp - kLoadWarp0);
    uint32_t issued = 0;
    bool ok = true;
#pragma unroll 1
    for (int ahead = 2; ahead > 0 || e0.live;) {  // pages are looked up two turns ahead
      e2.page = -1;
      e2.row = 0;
      e2.live = turns.next(walk, p);
      if (e2.live) {
        const int32_t pos = turns.step * kStep + lane * p.seg_rows;
        if (lane < segs && pos < walk.most) {
          const int32_t lb = pos >> p.page_shift;
          e2.row = (pos - (lb << p.page_shift)) / 2;  // a line holds two
          e2.page = __ldg(p.s.block_table + static_cast<int64_t>(walk.seq) * p.s.max_blocks + lb);
        }
        turns.done();
      }
      if (ahead > 0) {
        --ahead;
        e0 = e1;
        e1 = e2;
        continue;
      }
      ok = warp_wait(bar(Bars::kEmpty, at.stage), at.phase ^ 1u, abort_addr, lim);
      if (!ok) break;
      const uint32_t full = bar(Bars::kFull, at.stage);
      if (issuer) mbar_arrive_tx(full, kStepCodes);
      // a page that does not resolve: past the pool, zeros
      const int32_t page =
          static_cast<uint32_t>(e0.page) < static_cast<uint32_t>(past) ? e0.page : past;
      const uint32_t dst = stage0 + at.stage * kStageBytes;
#pragma unroll 1
      for (int i0 = 0; i0 < segs; i0 += 4) {
        int32_t z[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[i] = __shfl_sync(0xffffffffu, page, i0 + i);
          y[i] = __shfl_sync(0xffffffffu, e0.row, i0 + i);
        }
        if (issuer) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i0 + i < segs) tma_load_3d(dst + (i0 + i) * piece, &codes_map, y[i], z[i], full);
          }
        }
        __syncwarp();
      }
      e0 = e1;
      e1 = e2;
      at.advance(kCopyWarps);
      ++issued;
    }
    if (lane == 0) st_shared_u32(ctl + Bars::kIssued + 4 * (warp - kLoadWarp0), issued);
  } else if (p.seg_rows > 0 && warp < kScaleWarp0 + kScaleWarps) {
    // ----------------------------------------------- scales, tensor copies
    // Lane l has lines l, l + 32, .. of the step: the scales of each tile's
    // rows l, l + 32, .. are one 16-byte line of each K half's layout.
    constexpr int kLines = kScoreTile / 32;
    const bool issuer = elect_one();
    const uint8_t* scales = p.s.cache + static_cast<int64_t>(p.s.page_size) * kIndexCodes;
    const uint32_t stride = static_cast<uint32_t>(p.s.block_stride);
    const uint32_t in_page = static_cast<uint32_t>(p.s.page_size) - 1;
    struct Turn {  // a step of this warp's
      int32_t q, most, step;
      uint32_t it;  // number of the step among the CTA's
      uint32_t stage, phase;
      int32_t page;  // lane l: page l of those that the step touches, from `first` on
      int32_t first;
      bool live;
    };
    const int32_t step_pages = max(kStep >> p.page_shift, 1);
    Turns turns(warp - kScaleWarp0, kScaleWarps, p.stages);
    walk.t1 = 0;
    Turn later, then, now;
    later.live = then.live = now.live = false;
    uint4 vals[kLines];   // now's scales, of an even and an odd position
    uint32_t valid = 0;   // bit t + 2 i: position t of line l + 32 i resolves
    uint32_t committed = 0;
    bool ok = true;
    // A turn's page ids are loaded three turns ahead, its scales fetched into L2
    // two and loaded one turn ahead. Nothing is in flight at the fence, which
    // would wait for it.
#pragma unroll 1
    for (int ahead = 3; ahead > 0 || now.live; --ahead) {
      if (ahead <= 0) {
        const uint32_t stage = now.stage;
        ok = warp_wait(bar(Bars::kEmpty, stage), now.phase ^ 1u, abort_addr, lim);
        if (!ok) break;
        const bool whole = __all_sync(0xffffffffu, valid == (1u << 2 * kLines) - 1);
        if (!whole) {
#pragma unroll
          for (int i = 0; i < kLines; ++i) {
            if (!(valid >> 2 * i & 1u)) vals[i].x = vals[i].y = 0;
            if (!(valid >> 2 * i & 2u)) vals[i].z = vals[i].w = 0;
          }
        }
        const uint32_t to = stage0 + stage * kStageBytes + kStepCodes + lane * 16;
        st_shared_v4(to, vals[0].x, vals[1].x, vals[2].x, vals[3].x);
        st_shared_v4(to + 512, vals[0].y, vals[1].y, vals[2].y, vals[3].y);
        st_shared_v4(to + 1024, vals[0].z, vals[1].z, vals[2].z, vals[3].z);
        st_shared_v4(to + 1536, vals[0].w, vals[1].w, vals[2].w, vals[3].w);
#pragma unroll
        for (int t = 0; t < kStepTiles; ++t) {
          uint32_t mask[kLines] = {~0u, ~0u, ~0u, ~0u};
          if (!whole) {
#pragma unroll
            for (int i = 0; i < kLines; ++i)
              mask[i] = __ballot_sync(0xffffffffu, valid >> (2 * i + t) & 1u);
          }
          if (issuer)
            st_shared_v4(base + (now.it * kStepTiles + t) % kMaskRing * 16, mask[0], mask[1],
                         mask[2], mask[3]);
        }
        TopByte top;
#pragma unroll
        for (int i = 0; i < kLines; ++i)
          top.add(vals[i].x), top.add(vals[i].y), top.add(vals[i].z), top.add(vals[i].w);
        fence_proxy_async_cta();
        __syncwarp();
        if (issuer) {  // into tensor memory; the stage is full when they are there
#pragma unroll
          for (int t = 0; t < kStepTiles; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              copy_scales(tmem + sfa_col + (stage * kStepTiles + t) * 8 + h * 4,
                          scale_desc(stage0 + stage * kStageBytes + kStepCodes + t * kTileScales +
                                     h * 512));
          mma_commit(bar(Bars::kFull, stage));
        }
        ++committed;
        const uint32_t most = top.of_warp();
        if (lane < kStepTiles) p.s.smax[now.q * p.s.tiles + now.step * kStepTiles + lane] = most;
      }
      // the next turn's scales
      now = then;
      if (now.live) {
        valid = 0;
        // Positions that do not resolve or are not in use read some of page 0.
        const uint32_t mine =
            static_cast<uint32_t>(now.page) < static_cast<uint32_t>(p.s.num_blocks) ? now.page : ~0u;
        const uint32_t pos0 = static_cast<uint32_t>(now.step) * kStep + 2 * lane;
#pragma unroll
        for (int i = 0; i < kLines; ++i) {
          const uint32_t pos = pos0 + i * 64;
          const uint32_t page =
              __shfl_sync(0xffffffffu, mine, (pos >> p.page_shift) - static_cast<uint32_t>(now.first));
          const uint8_t* from = scales + static_cast<uint64_t>(page != ~0u ? page : 0u) * stride +
                                (pos & in_page) * kIndexScales;
          vals[i] = __ldg(reinterpret_cast<const uint4*>(from));
          const uint32_t most = page != ~0u ? now.most : 0u;
          valid |= (pos < most ? 1u << 2 * i : 0u) | (pos + 1 < most ? 2u << 2 * i : 0u);
        }
      }
      // the scales of the one after it, a line of 16 rows a lane
      then = later;
      if (then.live) {
        constexpr uint32_t kRows = 128 / kIndexScales;
        const uint32_t pos = static_cast<uint32_t>(then.step) * kStep + lane % (kStep / kRows) * kRows;
        const uint32_t page = __shfl_sync(0xffffffffu, then.page,
                                          (pos >> p.page_shift) - static_cast<uint32_t>(then.first));
        if (lane < kStep / kRows && page < static_cast<uint32_t>(p.s.num_blocks))
          prefetch_l2(scales + static_cast<uint64_t>(page) * stride + (pos & in_page) * kIndexScales);
      }
      // the page ids of the one after that
      later.live = turns.next(walk, p);
      if (later.live) {
        later.q = walk.q, later.most = walk.most;
        later.step = turns.step, later.it = turns.it;
        later.stage = turns.at.stage, later.phase = turns.at.phase;
        later.first = (turns.step * kStep) >> p.page_shift;
        later.page = -1;
        if (lane < step_pages && (later.first + lane) << p.page_shift < walk.most)
          later.page = __ldg(p.s.block_table + static_cast<int64_t>(walk.seq) * p.s.max_blocks +
                             later.first + lane);
        turns.done();
      }
    }
    if (lane == 0) st_shared_u32(ctl + Bars::kCommitted + 4 * (warp - kScaleWarp0), committed);
    if (issuer) {  // scale copies of an aborted CTA have completed
      mma_commit(bar(Bars::kScaleDrain, warp - kScaleWarp0));
      drain(bar(Bars::kScaleDrain, warp - kScaleWarp0), 0);
    }
    __syncwarp();
  } else if (warp < kLoadWarp0 + kLoadWarps) {
    // ---------------------------------------------- key loads, row by row
    // Warp w has positions 64 w .. of a step, two a lane; a step's copies are
    // one group.
    constexpr int kInFlight = 2;
    static_assert(stage_count(kChunks, kMaxGroup) > kInFlight, "stages");
    const int part = warp - kLoadWarp0;
    int32_t step = 0;
    walk.t1 = 0;
    bool more = true;
    // Lane l keeps the run and step of the l-th step of every 32.
    int32_t info_q = 0, info_step = 0;
    struct Entry {
      int32_t page[2], row[2];
      bool live;
    };
    uint32_t fetched = 0;
    auto fetch = [&](Entry& e) {
      if (more && step == walk.t1) {
        more = walk.next(p);
        step = walk.t0;
      }
      e.live = more;
      if (!more) return;
      if (lane == fetched % 32) info_q = walk.q, info_step = step;
      ++fetched;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int32_t pos = step * kStep + part * 64 + u * 32 + lane;
        const int32_t lb = pos / p.s.page_size;
        e.row[u] = pos - lb * p.s.page_size;
        e.page[u] = pos < walk.most
                        ? __ldg(p.s.block_table +
                                static_cast<int64_t>(walk.seq) * p.s.max_blocks + lb)
                        : -1;
      }
      ++step;
    };
    // Where the scales of this lane's position 32 u + lane of the part are.
    auto scales_at = [&](uint32_t stage, int u) {
      return stage0 + stage * kStageBytes + kStepCodes + (lane & 1) * kTileScales +
             (u * 16 + (lane >> 1)) * 16 + part * 4;
    };
    Ring at(p.stages), done(p.stages);
    auto publish = [&](uint32_t it) {  // this warp's positions of step `it` have landed
      const uint32_t stage = done.stage;
      done.advance(1);
      TopByte top;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        top.add(ld_shared_u32(scales_at(stage, u)));
        top.add(ld_shared_u32(scales_at(stage, u) + 512));
      }
      const uint32_t most = top.of_warp();
      const int32_t q = __shfl_sync(0xffffffffu, info_q, it % 32);
      const int32_t tile = __shfl_sync(0xffffffffu, info_step, it % 32) * kStepTiles;
      fence_proxy_async_cta();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Bars::kFull, stage));
      if (lane < kStepTiles)
        reinterpret_cast<uint8_t*>(p.s.smax + q * p.s.tiles + tile + lane)[part] =
            static_cast<uint8_t>(most);
    };
    Entry e0, e1, e2;
    e0.live = e1.live = false;
    uint32_t it = 0;
    bool ok = true;
#pragma unroll 1
    for (int ahead = 2; ahead > 0 || e0.live;) {
      fetch(e2);
      if (ahead > 0) {
        --ahead;
        e0 = e1;
        e1 = e2;
        continue;
      }
      const uint32_t stage = at.stage;
      ok = warp_wait(bar(Bars::kEmpty, stage), at.phase ^ 1u, abort_addr, lim);
      if (!ok) break;
      at.advance(1);
      uint32_t found[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool live = e0.page[u] >= 0 && e0.page[u] < p.s.num_blocks;
        found[u] = __ballot_sync(0xffffffffu, live);
        const int64_t page = live ? e0.page[u] * p.s.block_stride : 0;
        const int64_t codes = page + static_cast<int64_t>(e0.row[u]) * kIndexCodes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // eight positions each, four lanes a position
          const int r = i * 8 + (lane >> 2);
          const int64_t from = __shfl_sync(0xffffffffu, codes, r);
          cp_async16_z(stage0 + stage * kStageBytes + code_off(part * 64 + u * 32 + r, lane & 3),
                       p.s.cache + from + (lane & 3) * 16, (found[u] >> r) & 1u);
        }
        const uint8_t* sc = p.s.cache + page + static_cast<int64_t>(p.s.page_size) * kIndexCodes +
                            static_cast<int64_t>(e0.row[u]) * kIndexScales;
        cp_async4_z(scales_at(stage, u), sc, live);
        cp_async4_z(scales_at(stage, u) + 512, sc + 4, live);
      }
#pragma unroll
      for (int t = 0; t < kStepTiles; ++t) {  // lane l: position 2 l + t of the part
        const uint32_t x = 2 * lane + t;
        const uint32_t mask =
            __ballot_sync(0xffffffffu, (x < 32 ? found[0] : found[1]) >> (x & 31u) & 1u);
        if (lane == 0)
          st_shared_u32(base + ((it * kStepTiles + t) % kMaskRing * 4 + part) * 4, mask);
      }
      cp_async_commit();
      if (it >= kInFlight) {
        cp_async_wait<kInFlight>();
        publish(it - kInFlight);
      }
      e0 = e1;
      e1 = e2;
      ++it;
    }
    cp_async_wait<0>();
    if (ok) {
#pragma unroll 1
      for (uint32_t k = it > kInFlight ? it - kInFlight : 0; k < it; ++k) publish(k);
    }
  } else if (warp >= kMmaWarp0 && warp < kMmaWarp0 + kMmaWarps) {
    // ---------------------------------------------------------- MMA issue
    constexpr uint32_t idesc = score_idesc(kHeads);
    const int which = warp - kMmaWarp0;
    const uint32_t sfb0 = tmem + kSfbCol + static_cast<uint32_t>(which * p.group) * 8;
    uint32_t run = 0;
    uint32_t first = 0;  // number of the step's first unit
    int32_t wait = which;
    uint32_t turn = 0;   // steps of this warp's
    Ring at(p.stages);
    bool ok = true;
    const bool issuer = elect_one();
    // The first of these warps copies the queries, a run ahead of the MMAs.
    Walk ahead = walk;
    uint32_t copied = 0;  // runs
    auto copy_queries = [&]() {
      const uint32_t bytes = static_cast<uint32_t>(ahead.count) * kImage;
      const uint32_t to = bar(Bars::kQFull, copied & 1u);
      mbar_arrive_tx(to, bytes);
#pragma unroll 1
      for (int i = 0; i < ahead.count; ++i)
        tma_load_2d(q_image(copied & 1u) + i * kImage, &image_map, 0,
                    (ahead.q + i) * static_cast<int32_t>(kImage / kImageLine), to);
      ++copied;
    };
    if (which == 0 && ahead.next(p) && issuer) copy_queries();
#pragma unroll 1
    while (ok && walk.next(p)) {
      const int buf = run & 1;
      bool pending = which == 0 && ahead.next(p);
      ok = warp_wait(bar(Bars::kQFull, buf), (run >> 1) & 1u, abort_addr, lim);
      if (!ok) break;
      tc_fence_after();
      const uint32_t image = q_image(buf);
      if (issuer) {
#pragma unroll 1
        for (int i = 0; i < walk.count; ++i)
          for (int h = 0; h < 2; ++h)
            copy_scales(sfb0 + i * 8 + h * 4,
                        scale_desc(image + i * kImage + image_scales(kHeads) + h * 512));
        const uint64_t q0 = sw64_desc(image);
#pragma unroll 1
        for (int32_t step = walk.t0; step < walk.t1; ++step, first += walk.count, at.advance(1)) {
          if (pending &&
              mbar_ready(bar(Bars::kQEmpty, copied & 1u), ((copied >> 1) & 1u) ^ 1u)) {
            copy_queries();
            pending = false;
          }
          if (wait > 0) {  // the other warp's
            --wait;
            continue;
          }
          wait = kMmaWarps - 1;
          const uint32_t stage = at.stage;
          ok = wait_bar(bar(Bars::kFull, stage), at.phase, abort_addr, lim);
          if (!ok) break;
          tc_fence_after();
          const uint32_t src = stage0 + stage * kStageBytes;
          const uint32_t sfa = tmem + sfa_col + stage * kStepTiles * 8;
          if (p.seg_rows == 0) {  // copies row by row: the scales are still in shared memory
#pragma unroll
            for (int x = 0; x < 2 * kStepTiles; ++x)
              copy_scales(sfa + 4 * x, scale_desc(src + kStepCodes + 512 * x));
          }
          const uint64_t a = sw128_desc(src);
          // Steps are issued in order, which the parities of the slots rely on:
          // after the other warp's step before this one.
          if (kMmaWarps > 1 && (which > 0 || turn > 0)) {
            ok = wait_bar(bar(Bars::kTurn, which), (turn - (which == 0)) & 1u, abort_addr, lim);
            if (!ok) break;
          }
          ++turn;
#pragma unroll 1
          for (int i = 0; i < walk.count; ++i) {
            // a descriptor's address counts 16 bytes; a K step is 32 bytes, and
            // a tile's rows are one half of the 128-byte lines
            const uint64_t b = q0 + i * (kImage / 16);
            const uint32_t sfb = sfb0 + i * 8;
#pragma unroll
            for (int u = 0; u < kUnitSlots; ++u) {
              const uint32_t n = (first + i) * kUnitSlots + u, slot = n % kSlots;
              ok = wait_bar(bar(Bars::kDEmpty, slot), ((n / kSlots) & 1u) ^ 1u, abort_addr, lim);
              if (!ok) break;
              tc_fence_after();
              const uint32_t d = tmem + slot * kSlotCols;
#pragma unroll
              for (int t = 0; t < kSlotTiles; ++t) {
                const int tile = u * kSlotTiles + t;
                mma_fp4(d + t * kHeads, a + 4 * tile, b, idesc, sfa + 8 * tile, sfb, 0);
                mma_fp4(d + t * kHeads, a + 4 * tile + 2, b + 2, idesc, sfa + 8 * tile + 4, sfb + 4,
                        1);
              }
              mma_commit(bar(Bars::kDFull, slot));
            }
            if (!ok) break;
          }
          if (!ok) break;
          if (kMmaWarps > 1) mbar_arrive(bar(Bars::kTurn, which ^ 1));
          mma_commit(bar(Bars::kEmpty, stage));
        }
        mma_commit(bar(Bars::kQEmpty, buf));
        if (pending && ok) {
          ok = wait_bar(bar(Bars::kQEmpty, copied & 1u), ((copied >> 1) & 1u) ^ 1u, abort_addr, lim);
          if (ok) copy_queries();
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      ++run;
    }
    if (issuer) {  // copies of an aborted CTA have landed
#pragma unroll 1
      for (uint32_t k = copied > 2 ? copied - 2 : 0; k < copied; ++k)
        drain(bar(Bars::kQFull, k & 1u), (k >> 1) & 1u);
    }
    // everything this thread issued has completed before the CTA ends
    if (issuer) {
      mma_commit(bar(Bars::kDrain, which));
      drain(bar(Bars::kDrain, which), 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.seg_rows > 0 && tid == 32 * kLoadWarp0 && ld_shared_u32(abort_addr) != 0)
    drain_codes(ctl, static_cast<uint32_t>(p.stages));
  if (warp == kMmaWarp0) tmem_dealloc(tmem);
  if (tid == 0) p.s.status[blockIdx.x] = ld_shared_u32(abort_addr);
}

// Dynamic shared memory of score_kernel<chunks> with runs of up to `group`.
constexpr size_t score_smem(int chunks, int group) {
  return kStageBase + static_cast<size_t>(stage_count(chunks, group)) * kStageBytes +
         2 * static_cast<size_t>(group) * image_bytes(32 * chunks);
}
constexpr size_t most_score_smem(int chunks) {
  size_t most = 0;
  for (int group = 1; group <= kMaxGroup; ++group)
    most = score_smem(chunks, group) > most ? score_smem(chunks, group) : most;
  return most;
}

// The pool's codes as lines of 128 bytes (two rows), in 128-byte swizzle; false
// where the page size is no power of two or below 16: a step is then not made
// of pieces of pages with whole groups of eight lines.
bool codes_tensor(const SelectParams& s, CUtensorMap* map, int32_t* seg_rows) {
  const int32_t P = s.page_size;
  *seg_rows = 0;
  if (P < 16 || (P & (P - 1)) != 0) return false;
  EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr || s.num_blocks >= INT32_MAX || s.block_stride > UINT32_MAX) return false;
  const int32_t rows = P < kStep ? P : kStep;
  const cuuint64_t dims[3] = {2 * kIndexCodes, static_cast<cuuint64_t>(P / 2),
                              static_cast<cuuint64_t>(s.num_blocks)};
  const cuuint64_t strides[2] = {2 * kIndexCodes, static_cast<cuuint64_t>(s.block_stride)};
  const cuuint32_t box[3] = {2 * kIndexCodes, static_cast<cuuint32_t>(rows / 2), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  if (enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(s.cache), dims, strides, box,
          es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  *seg_rows = rows;
  return true;
}

template <int kChunks>
int32_t launch_chunks(ScoreParams& p, cudaStream_t stream) {
  constexpr int kImage = image_bytes(32 * kChunks);
  const size_t smem = score_smem(kChunks, p.group);
  constexpr size_t kMost = most_score_smem(kChunks);
  static_assert(kMost + 1024 <= kMaxSharedBytes, "shared memory");  // 1024 static ones
  // The limit is the process's: calls of other threads rely on it, so that it is
  // the same one in every call. Before the tensor maps: this call binds the
  // device's context to the host thread, which may have made no other yet, and
  // the driver's encoder needs it.
  if (cudaFuncSetAttribute(score_kernel<kChunks>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kMost)) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  codes_tensor(p.s, &map, &p.seg_rows);
  CUtensorMap images;  // a box is a query token's image
  {
    EncodeTiledFn enc = encode_tiled();
    constexpr int kLines = kImage / kImageLine;
    const cuuint64_t dims[2] = {kImageLine / 4, static_cast<cuuint64_t>(p.s.num_q) * kLines};
    const cuuint64_t strides[1] = {kImageLine};
    const cuuint32_t box[2] = {kImageLine / 4, kLines};
    const cuuint32_t es[2] = {1, 1};
    if (enc == nullptr ||
        enc(&images, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, p.s.images, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return NVFP4_MLA_ERR_LAUNCH;
  }
  encode_kernel<<<p.s.num_q, 32 * kChunks * kIndexScales, 0, stream>>>(
      p.s.q_index, p.s.weights, p.s.num_heads, 32 * kChunks, p.s.images);
  if (int32_t st = launch_status()) return st;
  cudaLaunchConfig_t launch = {};
  launch.gridDim = dim3(p.ctas);
  launch.blockDim = dim3(kScoreThreads);
  launch.dynamicSmemBytes = smem;
  launch.stream = stream;
  cudaLaunchAttribute attr[1];  // sets itself up while the queries are encoded
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  launch.attrs = attr;
  launch.numAttrs = 1;
  if (cudaLaunchKernelEx(&launch, score_kernel<kChunks>, p, map, images) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  return NVFP4_MLA_OK;
}

}  // namespace

size_t query_image_bytes(int32_t num_heads) {
  return static_cast<size_t>(image_bytes((num_heads + 31) / 32 * 32));
}

int32_t launch_scores(SelectParams& s, int num_sms, cudaStream_t stream) {
  ScoreParams p;
  const int chunks = (s.num_heads + 31) / 32;
  // Query tokens of a sequence share its key tiles: runs as long as there are
  // tokens per sequence, on average, and shared memory for their queries.
  const int32_t mean = s.num_q / s.num_seqs;
  p.group = s.group = mean < 1 ? 1 : mean > kMaxGroup ? kMaxGroup : mean;
  p.stages = stage_count(chunks, p.group);
  p.ctas = s.score_ctas = num_sms < kStatusWords ? num_sms : kStatusWords;
  p.s = s;
  p.page_shift = 0;
  while (p.page_shift < 20 && 1 << p.page_shift < s.page_size) ++p.page_shift;
  switch (chunks) {
    case 1: return launch_chunks<1>(p, stream);
    case 2: return launch_chunks<2>(p, stream);
    case 3: return launch_chunks<3>(p, stream);
    default: return launch_chunks<4>(p, stream);
  }
}

}  // namespace nvfp4_mla
