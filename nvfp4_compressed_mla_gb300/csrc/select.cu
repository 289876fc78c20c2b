// select.cu -- choosing the blocks of the context with the highest index scores.
//
// The choice is the one that 64-bit arithmetic makes. With a_i the fp32 score
// of block i, e_i its exact one and |a_i - e_i| <= eps for every i, let T be
// the k-th largest a. The k-th largest e then lies within eps of T, so a block
// with a_i > T + 2 eps is in and one with a_i < T - 2 eps is out; what lies
// between (mostly T's block alone) is scored again exactly: codes are small
// integers and the product of two E4M3 scales has 8 significant bits, so a dot
// product of 128 terms is an exact double (multiples of 2^-20 below 2^31), and
// only the weighted sum over the heads rounds, to 53 bits.
//
// The bound: a dot product's terms sum up, in magnitude, to at most
// 6 smax * |q^_j|_1 with smax the largest scale of the visible keys, so with
// M = 6 smax * sum_j |w_j| |q^_j|_1 the fp32 score is off by at most
// (kDotError + (heads / 8 + 8) 2^-24) M: heads are summed up in eight parts.
#include <math.h>

#include "select_common.cuh"

namespace nvfp4_mla {

long long decode_wait_cycles();

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kListCap = 1024;  // candidates ranked from shared memory
// Error of a dot product on the tensor cores, relative to the sum of its
// terms' magnitudes.
constexpr double kDotError = 64.0 / 16777216.0;

// Ordered integers: a < b as floats iff key(a) < key(b); no NaN, -0 = +0.
__device__ __forceinline__ uint32_t key32(float a) {
  const uint32_t u = __float_as_uint(a + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint64_t key64(double a) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(a + 0.0));
  return u >> 63 ? ~u : u | (1ull << 63);
}
constexpr uint64_t kLowest64 = 0x000FFFFFFFFFFFFFull;  // key64(-inf)

// An E2M1 code as an integer: twice its value.
__device__ __forceinline__ int32_t twice_e2m1(uint32_t code) {
  const int32_t m = static_cast<int32_t>((0xC8643210u >> (4 * (code & 7u))) & 15u);
  return code & 8u ? -m : m;
}
// Eight codes of a word -> two words of four signed bytes.
__device__ __forceinline__ void expand_codes(uint32_t w, uint32_t& a, uint32_t& b) {
  a = b = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a |= (static_cast<uint32_t>(twice_e2m1(w >> (4 * i))) & 0xFFu) << (8 * i);
    b |= (static_cast<uint32_t>(twice_e2m1(w >> (4 * i + 16))) & 0xFFu) << (8 * i);
  }
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return f16_bits_to_f32(static_cast<uint16_t>(e4m3x2_to_f16x2(static_cast<uint16_t>(byte))));
}

struct SelShared {
  uint32_t q_codes[NVFP4_MLA_MAX_HEADS * kIndexScales * 4];  // signed bytes, twice the values
  float q_scale[NVFP4_MLA_MAX_HEADS * kIndexScales];
  float w[NVFP4_MLA_MAX_HEADS];
  uint32_t hist[256];
  uint64_t cand_key[kListCap];
  int32_t cand[kListCap];
  double red[kSelWarps];
  float redf[kSelWarps];
  int32_t warp_sum[kSelWarps];
  int32_t warp_sum2[kSelWarps];
  uint32_t pick, rest, cand_n, in_n, failed;
};

__device__ __forceinline__ float block_score(const SelectParams& p, const float* row, int32_t b,
                                             int per, int32_t granules) {
  float a = __ldcg(row + static_cast<int64_t>(b) * per);
  for (int i = 1; i < per; ++i)
    if (static_cast<int64_t>(b) * per + i < granules)
      a = fmaxf(a, __ldcg(row + static_cast<int64_t>(b) * per + i));
  return a;
}

// Exact score of position `pos` as an ordered key, by one warp.
__device__ uint64_t exact_key(const SelectParams& p, const SelShared& sh, int32_t seq,
                              int32_t pos) {
  const int lane = threadIdx.x & 31;
  const IndexRow at = resolve_index_row(seq, pos, p.block_table, p.num_seqs, p.max_blocks,
                                        p.page_size, p.num_blocks, p.block_stride);
  if (at.page < 0) return kLowest64;
  const uint8_t* page = p.cache + at.page;
  const int g = lane & 7;
  const uint2 c = __ldg(reinterpret_cast<const uint2*>(
      page + static_cast<int64_t>(at.row) * kIndexCodes + g * 8));
  const float ks = scale_value(__ldg(page + static_cast<int64_t>(p.page_size) * kIndexCodes +
                                     static_cast<int64_t>(at.row) * kIndexScales + g) &
                               0x7Fu);
  uint32_t k[4];
  expand_codes(c.x, k[0], k[1]);
  expand_codes(c.y, k[2], k[3]);
  double sum = 0.0;
  for (int j0 = 0; j0 < p.num_heads; j0 += 4) {  // four heads, eight lanes each
    const int j = j0 + (lane >> 3);
    double d = 0.0;
    if (j < p.num_heads) {
      const uint32_t* q = sh.q_codes + (j * kIndexScales + g) * 4;
      int dot = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dot = __dp4a(static_cast<int>(q[i]), static_cast<int>(k[i]), dot);
      d = static_cast<double>(dot) * 0.25 *
          static_cast<double>(ks * sh.q_scale[j * kIndexScales + g]);
    }
    d += __shfl_xor_sync(0xffffffffu, d, 1);
    d += __shfl_xor_sync(0xffffffffu, d, 2);
    d += __shfl_xor_sync(0xffffffffu, d, 4);
    if (j < p.num_heads) sum += static_cast<double>(sh.w[j]) * (d < 0.0 ? 0.0 : d);
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
  return sum != sum ? kLowest64 : key64(sum);
}

// Exact key of block b, by one warp.
__device__ uint64_t exact_block_key(const SelectParams& p, const SelShared& sh, int32_t seq,
                                    int32_t b, int32_t seen) {
  uint64_t best = 0;
  const int64_t first = static_cast<int64_t>(b) * p.block;
  for (int64_t pos = first; pos < first + p.block && pos < seen; ++pos) {
    const uint64_t k = exact_key(p, sh, seq, static_cast<int32_t>(pos));
    best = best > k ? best : k;
  }
  return best;
}

__device__ __forceinline__ int block_sum(int v, int32_t* warp_sum) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, warp_sum[threadIdx.x & 31]);
}

// Threads with v set before this one, over the block; `total` gets all of them.
__device__ __forceinline__ int block_rank(bool v, int32_t* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t m = __ballot_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) warp_sum[warp] = __popc(m);
  __syncthreads();
  int w = warp_sum[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + __popc(m & ((1u << lane) - 1));
}

// With hist[256] filled: the digit of the `rank`-th largest value (rank >= 1)
// and its rank among the values with that digit. One warp.
__device__ __forceinline__ void find_digit(SelShared& sh, uint32_t rank) {
  const int lane = threadIdx.x & 31;
  uint32_t c[8], mine = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) mine += c[i] = sh.hist[255 - (lane * 8 + i)];
  uint32_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  uint32_t before = upto - mine;
  if (before < rank && rank <= upto) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (before < rank && rank <= before + c[i]) {
        sh.pick = 255 - (lane * 8 + i);
        sh.rest = rank - before;
      }
      before += c[i];
    }
  }
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  extern __shared__ uint8_t raw[];
  SelShared& sh = *reinterpret_cast<SelShared*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t t = blockIdx.x;
  const int64_t width = static_cast<int64_t>(p.num_select) * p.block;
  int32_t* out = p.topk_idx + t * width;
  const int32_t seq = __ldg(p.q_seq + t);
  const int32_t seen = visible_positions(p, seq, __ldg(p.q_pos + t));
  const int32_t blocks = blocks_of_positions(seen, p.block);

  if (tid == 0) sh.failed = 0;
  __syncthreads();
  for (int i = tid; i < p.score_ctas; i += kSelThreads)
    if (__ldcg(p.status + i) != 0) sh.failed = 1;
  __syncthreads();
  if (sh.failed) {
    for (int64_t i = tid; i < width; i += kSelThreads) out[i] = -2;
    return;
  }
  if (blocks <= p.num_select) {  // all of them
    for (int64_t i = tid; i < width; i += kSelThreads)
      out[i] = i < seen ? static_cast<int32_t>(i) : -1;
    return;
  }

  const int granule = min(p.block, kMaxGranule);
  const int per = p.block / granule;
  const int32_t granules = (seen + granule - 1) / granule;
  float* row = p.scores + t * p.score_stride;
  // The forced blocks are at both ends: k of the n between them are chosen.
  const int32_t b0 = p.sink, n = blocks - p.sink - p.recent;
  const int32_t k = p.num_select - p.sink - p.recent;

  float lo = INFINITY, hi = INFINITY;  // in: > hi; in question: lo .. hi
  int32_t ties = 0;                    // chosen ones of those at lo == hi, by index
  if (k > 0) {
    // k-th largest score
    uint32_t prefix = 0, rank = k;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) sh.hist[tid] = 0;
      __syncthreads();
      for (int32_t i = tid; i < n; i += kSelThreads) {
        const uint32_t key = key32(block_score(p, row, b0 + i, per, granules));
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&sh.hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) find_digit(sh, rank);
      __syncthreads();
      prefix |= sh.pick << shift;
      rank = sh.rest;
      __syncthreads();
    }
    const float T = unkey32(prefix);

    // the heads as integers, and the error bound
    double m = 0.0;
    for (int g = tid; g < p.num_heads * kIndexScales; g += kSelThreads) {
      const uint8_t* src =
          p.q_index + (static_cast<int64_t>(t) * p.num_heads * kIndexScales + g) * (2 * kGroup);
      const uint4 a = ld_nc_v4(src), b = ld_nc_v4(src + 16);
      const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t c0, c1;
      float s;
      quantize_group(v, c0, c1, s);
      uint32_t e[4];
      expand_codes(c0, e[0], e[1]);
      expand_codes(c1, e[2], e[3]);
      int mag = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sh.q_codes[g * 4 + i] = e[i];
        mag = __dp4a(static_cast<int>(__vabs4(e[i])), 0x01010101, mag);
      }
      sh.q_scale[g] = s;
      const float w = __ldg(p.weights + static_cast<int64_t>(t) * p.num_heads + g / kIndexScales);
      if (g % kIndexScales == 0) sh.w[g / kIndexScales] = w;
      m += static_cast<double>(fabsf(w)) * (0.5 * mag) * static_cast<double>(s);
    }
    int32_t lead = t;  // first token of t's run
    while (lead % p.group != 0 && __ldg(p.q_seq + lead - 1) == seq) --lead;
    uint32_t top = 0;
    const int32_t tiles = (seen + kScoreTile - 1) / kScoreTile;
    for (int32_t i = tid; i < tiles; i += kSelThreads)
      top = __vmaxu4(top, __ldcg(p.smax + lead * p.tiles + i));
    top = __vmaxu4(top, top >> 16);
    top = __vmaxu4(top, top >> 8) & 0xFFu;
    float smax = scale_value(top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      m += __shfl_xor_sync(0xffffffffu, m, d);
      smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, d));
    }
    if (lane == 0) sh.red[warp] = m, sh.redf[warp] = smax;
    __syncthreads();
    m = sh.red[lane];
    smax = sh.redf[lane];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      m += __shfl_xor_sync(0xffffffffu, m, d);
      smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, d));
    }
    m *= 6.0 * static_cast<double>(smax);
    // rounded up to fp32; the last term covers products below the smallest
    // normal fp32
    const double eps = m == 0.0 ? 0.0 : m * (kDotError + (p.num_heads / 8 + 8) / 16777216.0) + 1e-40;
    const float eps2 = __double2float_ru(2.0 * eps);
    // A score of -inf comes from a NaN or a page that does not resolve, not
    // from rounding, unless fp32 overflowed.
    const bool bounded = m < 1e37;
    if (bounded && (eps2 == 0.f || T == -INFINITY)) {
      lo = hi = T;
      ties = static_cast<int32_t>(rank);
    } else {
      lo = bounded ? __fadd_rd(T, -eps2) : -INFINITY;
      hi = bounded ? __fadd_ru(T, eps2) : INFINITY;
      // candidates
      if (tid == 0) sh.cand_n = 0;
      __syncthreads();
      int in = 0;
      for (int32_t i = tid; i < n; i += kSelThreads) {
        const float a = block_score(p, row, b0 + i, per, granules);
        if (a > hi) {
          ++in;
        } else if (a >= lo) {
          const uint32_t c = atomicAdd(&sh.cand_n, 1u);
          if (c < kListCap) sh.cand[c] = b0 + i;
        }
      }
      in = block_sum(in, sh.warp_sum);
      const int32_t cands = static_cast<int32_t>(sh.cand_n);
      const int32_t want = k - in;  // 1 <= want <= cands
      if (cands == want) {
        ties = want;  // all of them
      } else if (cands <= kListCap) {
        for (int i = tid; i < cands; i += kSelThreads) sh.cand_key[i] = 0;
        __syncthreads();
        for (int64_t i = warp; i < static_cast<int64_t>(cands) * p.block; i += kSelWarps) {
          const int c = static_cast<int>(i / p.block);
          const int64_t pos = static_cast<int64_t>(sh.cand[c]) * p.block + i % p.block;
          if (pos >= seen) continue;
          const uint64_t key = exact_key(p, sh, seq, static_cast<int32_t>(pos));
          if (lane == 0)
            atomicMax(reinterpret_cast<unsigned long long*>(&sh.cand_key[c]),
                      static_cast<unsigned long long>(key));
        }
        __syncthreads();
        for (int i = tid; i < cands; i += kSelThreads) {
          const uint64_t key = sh.cand_key[i];
          const int32_t b = sh.cand[i];
          int better = 0;
          for (int j = 0; j < cands; ++j)
            better += sh.cand_key[j] > key || (sh.cand_key[j] == key && sh.cand[j] < b);
          float* at = row + static_cast<int64_t>(b) * per;
          for (int g = 0; g < per && static_cast<int64_t>(b) * per + g < granules; ++g)
            at[g] = better < want ? INFINITY : -INFINITY;
        }
        hi = fminf(hi, 3.402823466e38f);  // below +inf, the chosen ones' mark
        __syncthreads();
      } else {
        // Too many to list: radix selection on the exact keys, computed anew
        // for each digit; then candidates above the border become +inf, those
        // on it NaN-free ties at the largest finite value, the others -inf.
        uint64_t edge = 0;
        uint32_t left = want;
        for (int shift = 56; shift >= 0; shift -= 8) {
          if (tid < 256) sh.hist[tid] = 0;
          __syncthreads();
          for (int32_t i = warp; i < n; i += kSelWarps) {
            const float a = block_score(p, row, b0 + i, per, granules);
            if (!(a >= lo && a <= hi)) continue;
            const uint64_t key = exact_block_key(p, sh, seq, b0 + i, seen);
            if (lane == 0 && (shift == 56 || (key >> (shift + 8)) == (edge >> (shift + 8))))
              atomicAdd(&sh.hist[(key >> shift) & 255u], 1u);
          }
          __syncthreads();
          if (warp == 0) find_digit(sh, left);
          __syncthreads();
          edge |= static_cast<uint64_t>(sh.pick) << shift;
          left = sh.rest;
          __syncthreads();
        }
        for (int32_t i = warp; i < n; i += kSelWarps) {
          const float a = block_score(p, row, b0 + i, per, granules);
          if (a > hi) {
            // in: above any tie
          } else if (!(a >= lo)) {
            continue;
          }
          const uint64_t key = a > hi ? ~0ull : exact_block_key(p, sh, seq, b0 + i, seen);
          __syncwarp();
          if (lane == 0) {
            float* at = row + static_cast<int64_t>(b0 + i) * per;
            for (int g = 0; g < per && static_cast<int64_t>(b0 + i) * per + g < granules; ++g)
              at[g] = key > edge ? INFINITY : key == edge ? 3.402823466e38f : -INFINITY;
          }
          __syncwarp();
        }
        lo = hi = 3.402823466e38f;
        ties = static_cast<int32_t>(left);
        __syncthreads();
      }
    }
  }

  // Blocks in order: chosen ones get the next row of the output. A block is in
  // above hi, and among the first `ties` at lo .. hi.
  int32_t done = 0, ties_seen = 0;
  for (int32_t c0 = 0; c0 < blocks; c0 += kSelThreads) {
    const int32_t b = c0 + tid;
    const bool forced = b < blocks && (b < p.sink || b >= blocks - p.recent);
    bool in = forced, tie = false;
    if (b < blocks && !forced && k > 0) {
      const float a = block_score(p, row, b, per, granules);
      in = a > hi;
      tie = !in && a >= lo;
    }
    int total;
    if (ties > 0) {
      const int r = block_rank(tie, sh.warp_sum, total);
      in = in || (tie && ties_seen + r < ties);
      ties_seen += total;
    }
    const int r = block_rank(in, sh.warp_sum2, total);
    if (in) out[static_cast<int64_t>(done + r) * p.block] = b * p.block;
    done += total;
  }
  __syncthreads();
  // Each block's first position is in place: the others follow from it.
  if (p.block > 1) {
    for (int64_t i = tid; i < width; i += kSelThreads) {
      const int off = static_cast<int>(i % p.block);
      if (off == 0) continue;
      const int32_t pos = __ldcg(out + (i - off)) + off;
      out[i] = pos < seen ? pos : -1;
    }
  }
}

struct Workspace {
  int64_t score_stride, tiles;
  size_t per_q, bytes;
  int32_t chunk;
};

constexpr size_t kWorkspaceGoal = size_t{256} << 20;

bool plan_workspace(int32_t num_q, int32_t num_heads, int32_t max_blocks, int32_t page_size,
                    int32_t block, Workspace& w) {
  if (num_q < 0 || num_heads < 1 || num_heads > NVFP4_MLA_MAX_HEADS || max_blocks < 1 ||
      page_size < 1 || page_size > (1 << 20) || page_size % 2 != 0 ||
      static_cast<int64_t>(max_blocks) * page_size > INT32_MAX - 511 || block < 1 ||
      block > kScoreTile || (block & (block - 1)) != 0)
    return false;
  const int64_t room = static_cast<int64_t>(max_blocks) * page_size;
  const int64_t granule = block < kMaxGranule ? block : kMaxGranule;
  w.score_stride = ((room + granule - 1) / granule + 3) / 4 * 4;
  w.tiles = ((room + kScoreTile - 1) / kScoreTile + 3) / 4 * 4;
  w.per_q = static_cast<size_t>(w.score_stride + w.tiles) * 4;
  size_t fit = kWorkspaceGoal / w.per_q;
  if (fit < 1) fit = 1;
  if (fit > 32768) fit = 32768;
  w.chunk = num_q < static_cast<int64_t>(fit) ? num_q : static_cast<int32_t>(fit);
  w.bytes = num_q == 0 ? 0 : w.per_q * w.chunk + kStatusWords * 4;
  return true;
}

}  // namespace
}  // namespace nvfp4_mla

using namespace nvfp4_mla;

extern "C" size_t sparse_mla_select_workspace_size(int32_t num_q, int32_t num_heads,
                                                   int32_t max_blocks_per_seq, int32_t page_size,
                                                   int32_t select_block) {
  Workspace w;
  if (!plan_workspace(num_q, num_heads, max_blocks_per_seq, page_size, select_block, w))
    return SIZE_MAX;
  return w.bytes;
}

extern "C" int32_t sparse_mla_select(const void* q_index, const float* weights,
                                     const int32_t* q_seq, const int32_t* q_pos, int32_t num_q,
                                     int32_t num_heads, const int32_t* block_table,
                                     int32_t num_seqs, int32_t max_blocks_per_seq,
                                     int32_t page_size, const void* cache, int64_t num_blocks,
                                     int64_t block_stride_bytes, int32_t select_block,
                                     int32_t num_select, int32_t sink_blocks,
                                     int32_t recent_blocks, int32_t* topk_idx, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  Workspace w;
  if (!plan_workspace(num_q, num_heads, max_blocks_per_seq, page_size, select_block, w) ||
      num_select < 1 ||
      static_cast<int64_t>(num_select) * select_block > NVFP4_MLA_MAX_TOPK || sink_blocks < 0 ||
      recent_blocks < 0 || static_cast<int64_t>(sink_blocks) + recent_blocks > num_select)
    return NVFP4_MLA_ERR_SHAPE;
  if (num_q == 0) return NVFP4_MLA_OK;
  if (!q_index || !weights || !q_seq || !q_pos || !block_table || !cache || !topk_idx)
    return NVFP4_MLA_ERR_NULL;
  if (!index_shape_ok(num_seqs, max_blocks_per_seq, page_size, num_blocks, block_stride_bytes))
    return NVFP4_MLA_ERR_SHAPE;
  if (!aligned16(q_index) || !aligned16(cache) || (block_stride_bytes & 15))
    return NVFP4_MLA_ERR_ALIGN;
  if (!workspace || workspace_bytes < w.bytes) return NVFP4_MLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return NVFP4_MLA_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;
  if (cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sizeof(SelShared))) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t q0 = 0; q0 < num_q; q0 += w.chunk) {
    SelectParams p = {};
    p.num_q = num_q - q0 < w.chunk ? num_q - q0 : w.chunk;
    p.num_heads = num_heads;
    p.q_index = static_cast<const uint8_t*>(q_index) +
                static_cast<int64_t>(q0) * num_heads * kIndexDim * 2;
    p.weights = weights + static_cast<int64_t>(q0) * num_heads;
    p.q_seq = q_seq + q0;
    p.q_pos = q_pos + q0;
    p.block_table = block_table;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.page_size = page_size;
    p.cache = static_cast<const uint8_t*>(cache);
    p.num_blocks = num_blocks;
    p.block_stride = block_stride_bytes;
    p.block = select_block;
    p.num_select = num_select;
    p.sink = sink_blocks;
    p.recent = recent_blocks;
    p.topk_idx = topk_idx + static_cast<int64_t>(q0) * num_select * select_block;
    p.scores = static_cast<float*>(workspace);
    p.score_stride = w.score_stride;
    p.smax = reinterpret_cast<uint32_t*>(p.scores + w.score_stride * w.chunk);
    p.tiles = w.tiles;
    p.status = reinterpret_cast<uint32_t*>(p.smax + w.tiles * w.chunk);
    p.wait_cycles = decode_wait_cycles();
    if (int32_t st = launch_scores(p, sms, s)) return st;
    select_kernel<<<p.num_q, kSelThreads, sizeof(SelShared), s>>>(p);
    if (int32_t st = launch_status()) return st;
  }
  return NVFP4_MLA_OK;
}
