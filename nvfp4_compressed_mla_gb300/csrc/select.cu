// select.cu -- choosing the blocks of the context with the highest index scores.
//
// The choice is the one that 64-bit arithmetic makes. With a_i the fp32 score
// of block i, e_i its exact one and |a_i - e_i| <= eps for every i, let T be
// the k-th largest a. The k-th largest e then lies within eps of T, so a block
// with a_i > T + 2 eps is in and one with a_i < T - 2 eps is out; what lies
// between (mostly T's block and a few neighbours) is scored again: codes are
// small integers and the product of two E4M3 scales has 8 significant bits, so
// a dot product of 128 terms is an exact 51-bit integer. Summed up over the
// heads in fp32 that gives an interval around e_i a thousand times narrower
// than 2 eps; blocks whose intervals still overlap at the border are summed up
// in fp64, which this part runs at 1/64 of its fp32 rate.
//
// The bound: a dot product's terms sum up, in magnitude, to at most
// 6 smax * |q^_j|_1 with smax the largest scale of the visible keys, so with
// M = 6 smax * sum_j |w_j| |q^_j|_1 the fp32 score is off by at most
// (kDotError + (heads / 8 + 4) 2^-24) M: heads are summed up in eight parts.
//
// One CTA per query token holds the scores of all blocks in shared memory
// where they fit (16384; 32768 beside tables of more than 2^19 blocks). Longer
// rows: a sample of 4096 scores gives a
// threshold that a little more than k of them pass, one sweep collects those
// that do (a cluster of CTAs shares the sweep where there are few query
// tokens), and the choice is made among them. Where a sweep collects too few
// or too many, and for a border among equal scores, the general form reads the
// scores from memory in every step.
//
// A chain of phases of 1 to 10 us, bound by the latency of their loads, of shared
// memory atomics and of barriers; no unit is near its limit. Measured (GB300,
// device time, beginning beside the end of the scoring): 1 row of 4096 scores,
// 256 chosen, 15 us; 66 rows of about 146000, 2048 chosen, 54 us; as many of
// 2300 blocks of 64, 32 us; 480 rows of 65536 121 us; 2048 rows of 1024 blocks
// of 16 80 us; 1 row of a million 60 us.
#include <math.h>

#include "select_common.cuh"

namespace nvfp4_mla {

long long decode_wait_cycles();

namespace {

constexpr int kBins = 2048;
// 2048 leave more to collect: 66 rows of 146000 scores 0.7 us less, 480 rows of
// 65536 2 us more.
constexpr int kSample = 4096;
// Keys that a CTA holds: all of a row's, or the keys and blocks of half as
// many collected ones, or a bit for each of 32 times as many blocks.
constexpr int kRoom = 16384, kWideRoom = 32768;
constexpr int kMaxCluster = 8;
// Error of a dot product on the tensor cores, relative to the sum of its
// terms' magnitudes: 2.9 x 2^-24 is the most measured over 5e5 dot products,
// with scales up to 2^15 apart.
constexpr float kDotError = 8.0f / 16777216.0f;
// Error of an fp32 sum over the heads of exact dot products, relative to
// sum_j |w_j| D_j: two roundings of each D, at most four terms and
// five shuffles in a chain, and those of the bound itself.
constexpr float kSumError = 16.0f / 16777216.0f;
constexpr float kTiny = 1e-42f;  // products below the smallest normal fp32 round by less

// Ordered integers: a < b as floats iff key(a) < key(b); -0 = +0. The keys of
// NaNs mark blocks whose fate is known.
constexpr uint32_t kIn = 0xFFFFFFFFu, kTie = 0xFFFFFFFEu, kOut = 0u;
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
__device__ __forceinline__ uint32_t load_volatile(const uint32_t* at) {
  return *static_cast<const volatile uint32_t*>(at);
}
constexpr uint64_t kLowest64 = 0x000FFFFFFFFFFFFFull;  // key64(-inf)

// An E2M1 code as an integer: twice its value.
__device__ __forceinline__ int32_t twice_e2m1(uint32_t code) {
  const int32_t m = static_cast<int32_t>((0xC8643210u >> (4 * (code & 7u))) & 15u);
  return code & 8u ? -m : m;
}
// Four codes -> four signed bytes.
__device__ __forceinline__ uint32_t expand_codes(uint32_t w) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a |= (static_cast<uint32_t>(twice_e2m1(w >> (4 * i))) & 0xFFu) << (8 * i);
  return a;
}
// An E4M3 scale byte as an integer m * 2^s, in units of 2^-9: m | s << 8.
__device__ __forceinline__ uint32_t scale_parts(uint32_t byte) {
  const uint32_t e = byte >> 3 & 15u, m = byte & 7u;
  return e != 0 ? (8u + m) | (e - 1) << 8 : m;
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return f16_bits_to_f32(static_cast<uint16_t>(e4m3x2_to_f16x2(static_cast<uint16_t>(byte))));
}

constexpr int kTokens = 4;                     // that a warp scores at a time
template <int kN>
struct Count {
  static constexpr int value = kN;
};
constexpr int kStageWords = kTokens * (32 + 8);  // their codes and scales

template <int kThreads>
struct SelShared {
  static constexpr int kWarps = kThreads / 32;
  static constexpr int kCands = kThreads;  // candidates ranked from shared memory
  uint4 q_codes[kIndexScales][NVFP4_MLA_MAX_HEADS];  // signed bytes, twice the values
  uint4 stage[kWarps][kStageWords / 4];
  uint16_t q_scale[kIndexScales][NVFP4_MLA_MAX_HEADS];
  float w[NVFP4_MLA_MAX_HEADS];
  uint32_t hist[kBins];
  uint64_t cand_key[kCands];              // fp64 score, as a key
  uint32_t cand_lo[kCands], cand_hi[kCands];  // interval around the exact score, as keys
  int32_t cand[kCands];                   // position in the row of keys
  float red[kWarps];
  uint32_t redu[kWarps], redv[kWarps];
  int32_t sum_a[kWarps], sum_b[kWarps];
  uint32_t pick, rest, n, failed;
};

struct SelectConfig {
  int32_t room;  // keys that the dynamic shared memory behind SelShared holds
};

// ------------------------------------------------------------- block helpers
template <int kThreads>
__device__ __forceinline__ int block_sum(int v, int32_t* sums) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? sums[lane] : 0);
}

// Sum of v over the threads before this one; `total` gets that over all.
template <int kThreads>
__device__ __forceinline__ int block_before(int v, int32_t* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int w = lane < kThreads / 32 ? sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < kThreads / 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, kThreads / 32 - 1);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + upto - v;
}

// With hist filled: the bin of the `rank`-th largest value (rank >= 1) into
// sh.pick and its rank among that bin's values into sh.rest.
template <int kThreads>
__device__ __forceinline__ void find_bin(SelShared<kThreads>& sh, uint32_t rank) {
  constexpr int kPer = kBins / kThreads;
  const int top = kBins - 1 - static_cast<int>(threadIdx.x) * kPer;  // this thread's highest bin
  uint32_t c[kPer];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine += c[i] = sh.hist[top - i];
  int total;
  uint32_t before = block_before<kThreads>(mine, sh.sum_a, total);
  if (before < rank && rank <= before + mine) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (before < rank && rank <= before + c[i]) sh.pick = top - i, sh.rest = rank - before;
      before += c[i];
    }
  }
  __syncthreads();
}

// The `rank`-th largest of `count` keys: a histogram over their range, then
// over the bin that holds it, until a bin is one value (three levels for fp32
// keys, which differ in 22 to 32 bits). each(f) calls f with this thread's
// share of the keys, and the whole block goes through it; `rank` becomes the
// rank among the equal ones. With fewer levels the lower edge of the last bin.
template <int kThreads, typename Key, int kLevels = 8, typename Each>
__device__ __forceinline__ Key kth_largest(SelShared<kThreads>& sh, Key lowest, Key highest,
                                           uint32_t& rank, Each&& each) {
  Key base = lowest, width = highest - lowest;  // keys base .. base + width are in question
  for (int level = 1;; ++level) {
    const int bits = width == 0 ? 0 : sizeof(Key) == 8
                                          ? 64 - __clzll(static_cast<long long>(width))
                                          : 32 - __clz(static_cast<int>(width));
    const int shift = bits > 11 ? bits - 11 : 0;
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    each([&](Key k) {
      if (k >= base && k - base <= width) atomicAdd(&sh.hist[(k - base) >> shift], 1u);
    });
    __syncthreads();
    find_bin<kThreads>(sh, rank);
    base += static_cast<Key>(sh.pick) << shift;
    rank = sh.rest;
    __syncthreads();
    if (shift == 0 || level == kLevels) return base;
    width = (Key{1} << shift) - 1;
  }
}

// Lowest and highest of the keys that each() goes through.
template <int kThreads, typename Each>
__device__ __forceinline__ void key_range(SelShared<kThreads>& sh, uint32_t& lowest,
                                          uint32_t& highest, Each&& each) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  each([&](uint32_t k) { lo = min(lo, k), hi = max(hi, k); });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __syncthreads();
  if (lane == 0) sh.redu[warp] = lo, sh.redv[warp] = hi;
  __syncthreads();
  constexpr int kW = kThreads / 32;
  lowest = __reduce_min_sync(0xffffffffu, sh.redu[lane % kW]);
  highest = __reduce_max_sync(0xffffffffu, sh.redv[lane % kW]);
}

// ------------------------------------------------------------ exact scores
// Dot products of `n` consecutive positions (1 .. kTok) with all heads as
// exact integers in units of 2^-20, lane = head, 32 heads at a time, and their
// weighted sums: in fp32 with an error bound, or in fp64. One warp; the keys go
// through shared memory, where a 16-byte broadcast serves 16 codes, and the
// heads' codes are read once for all the positions.
// Where the fp32 sum of the magnitudes overflows (or a weight is not finite), the error
// is not finite, and the value says nothing.
struct TokenScore {
  float value, error;
  double exact;
  bool none;  // -inf: a NaN, or a page that does not resolve
};
template <bool kExact, int kTok, int kThreads>
__device__ __forceinline__ void score_tokens(const SelectParams& p, SelShared<kThreads>& sh,
                                             int32_t seq, int32_t pos, int n,
                                             TokenScore (&r)[kTok]) {
  const int lane = threadIdx.x & 31;
  uint4* codes = sh.stage[threadIdx.x >> 5];
  uint32_t* scales = reinterpret_cast<uint32_t*>(codes + kTokens * 8);
  const IndexRow at =
      resolve_index_row(seq, pos + min(lane & (kTok - 1), n - 1), p.block_table, p.num_seqs,
                        p.max_blocks, p.page_size, p.num_blocks, p.block_stride);
  uint32_t word[kTok], byte[kTok];
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    const int64_t page = __shfl_sync(0xffffffffu, static_cast<int64_t>(at.page), t);
    const int64_t row = __shfl_sync(0xffffffffu, at.row, t);
    word[t] = 0, byte[t] = 0x7Fu;
    if (t < n && page >= 0) {
      const uint8_t* base = p.cache + page;
      word[t] = __ldg(reinterpret_cast<const uint16_t*>(base + row * kIndexCodes + lane * 2));
      byte[t] = __ldg(base + static_cast<int64_t>(p.page_size) * kIndexCodes + row * kIndexScales +
                      (lane & 7)) &
                0x7Fu;
    }
  }
  __syncwarp();
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    r[t] = {0.f, 0.f, 0.0, __any_sync(0xffffffffu, byte[t] == 0x7Fu) != 0};
    if (t < n) {
      reinterpret_cast<uint32_t*>(codes)[t * 32 + lane] = expand_codes(word[t]);
      if (lane < 8) scales[t * 8 + lane] = scale_parts(byte[t]);
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int j0 = 0; j0 < p.num_heads; j0 += 32) {
    const int j = min(j0 + lane, p.num_heads - 1);
    int64_t d[kTok] = {};
#pragma unroll(kTok == 1 ? kIndexScales : 2)
    for (int g = 0; g < kIndexScales; ++g) {
      const uint4 q = sh.q_codes[g][j];
      const uint32_t qs = sh.q_scale[g][j];
#pragma unroll
      for (int t = 0; t < kTok; ++t) {
        if (t >= n) break;
        const uint4 k = codes[t * 8 + g];
        const uint32_t ks = scales[t * 8 + g];
        int dot = __dp4a(static_cast<int>(q.x), static_cast<int>(k.x), 0);
        dot = __dp4a(static_cast<int>(q.y), static_cast<int>(k.y), dot);
        dot = __dp4a(static_cast<int>(q.z), static_cast<int>(k.z), dot);
        dot = __dp4a(static_cast<int>(q.w), static_cast<int>(k.w), dot);
        dot *= static_cast<int>((ks & 255u) * (qs & 255u));
        d[t] += static_cast<int64_t>(dot) << ((ks >> 8) + (qs >> 8));
      }
    }
    const float w = sh.w[j];
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      if (t >= n) break;
      if (d[t] < 0 || j0 + lane >= p.num_heads) d[t] = 0;
      if (kExact) {
        // most weights of zero dot products need no fp64
        if (__any_sync(0xffffffffu, d[t] > 0))
          r[t].exact += static_cast<double>(w) * (static_cast<double>(d[t]) * 0x1p-20);
      } else {
        const float f = fmaf(static_cast<float>(static_cast<int32_t>(d[t] >> 24)), 16777216.f,
                             static_cast<float>(static_cast<int32_t>(d[t] & 0xFFFFFF))) *
                        0x1p-20f;
        r[t].value = fmaf(w, f, r[t].value);
        r[t].error = fmaf(fabsf(w), f, r[t].error);
        if (f > 0.f && w != 0.f) r[t].error += kTiny;  // never 0 by underflow
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    if (t >= n) break;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      if (kExact) {
        r[t].exact += __shfl_xor_sync(0xffffffffu, r[t].exact, s);
      } else {
        r[t].value += __shfl_xor_sync(0xffffffffu, r[t].value, s);
        r[t].error += __shfl_xor_sync(0xffffffffu, r[t].error, s);
      }
    }
    if (kExact) {
      r[t].none = r[t].none || r[t].exact != r[t].exact;
    } else {
      r[t].error = r[t].error == 0.f ? 0.f : __fadd_ru(__fmul_ru(r[t].error, kSumError), kTiny);
    }
  }
}
// Raises the bounds of a block's highest score by those of `n` consecutive
// positions. A score that fp32 does not bound may be anything: fp64 tells.
template <int kTok, int kThreads>
__device__ __forceinline__ void widen(const SelectParams& p, SelShared<kThreads>& sh, int32_t seq,
                                      int32_t pos, int n, float& low, float& high) {
  TokenScore r[kTok];
  score_tokens<false, kTok>(p, sh, seq, pos, n, r);
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    if (t >= n) break;
    if (r[t].none) continue;
    if (r[t].error < INFINITY) {
      low = fmaxf(low, __fsub_rd(r[t].value, r[t].error));
      high = fmaxf(high, __fadd_ru(r[t].value, r[t].error));
    } else {
      high = INFINITY;
    }
  }
}
// The highest fp64 score of `n` consecutive positions, as a key.
template <int kTok, int kThreads>
__device__ __forceinline__ uint64_t exact_key(const SelectParams& p, SelShared<kThreads>& sh,
                                              int32_t seq, int32_t pos, int n) {
  TokenScore r[kTok];
  score_tokens<true, kTok>(p, sh, seq, pos, n, r);
  uint64_t best = 0;
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    if (t >= n) break;
    const uint64_t key = r[t].none ? kLowest64 : key64(r[t].exact);
    best = best > key ? best : key;
  }
  return best;
}

// ------------------------------------------------------------- the choice
// Who is in, in terms of a row's keys: above `hi`, and of those at lo .. hi
// the first `ties` by index.
struct Border {
  uint32_t lo, hi;
  int32_t ties;
};

// The border where more scores lie next to it than can be listed, mostly among
// equal ones: the want-th largest of the keys lo .. hi.
template <int kThreads, typename Row>
__device__ __forceinline__ Border choose_unlisted(const SelectParams& p, SelShared<kThreads>& sh,
                                               const Row& row, int32_t count, int32_t want,
                                               int32_t seq, int32_t seen, uint32_t lo,
                                               uint32_t hi) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  const int per_piece = min(p.block, kTokens);
  auto pieces = [&](int32_t i, auto&& each) {  // until each() is false; one warp
    const int64_t first = static_cast<int64_t>(row.block(i)) * p.block;
#pragma unroll 1
    for (int64_t pos = first; pos < first + p.block && pos < seen; pos += per_piece)
      if (!each(static_cast<int32_t>(pos), min(per_piece, seen - static_cast<int32_t>(pos)))) break;
  };
  // Scores of 0 are exact in fp32: where the border lies among them, one pass
  // tells who is above and who is equal.
  const bool capped =
      __syncthreads_or(tid < p.num_heads && sh.w[min(tid, p.num_heads - 1)] > 0.f) == 0;
  if (lo <= key32(0.f) && key32(0.f) <= hi) {
    int above = 0, equal = 0, open = 0;
    int zeros = 0;     // capped: found so far by all warps, and
    bool sure = true;  // nothing undecided before them
#pragma unroll 1
    for (int32_t i0 = 0; i0 < count; i0 += kWarps) {
      const int32_t i = i0 + warp;
      const uint32_t key = i < count ? row.key(i) : kOut;
      bool tie = false, unknown = false;
      if (key >= lo && key <= hi) {
        float low = -INFINITY, high = -INFINITY;
        pieces(i, [&](int32_t pos, int of) {
          widen<kTokens>(p, sh, seq, pos, of, low, high);
          return !(capped && low == 0.f);
        });
        if (capped) high = fminf(high, 0.f);
        __syncwarp();
        const bool in = low > 0.f, out = high < 0.f;
        tie = low == 0.f && high == 0.f;
        unknown = !(in || out || tie);
        if (lane == 0) {
          above += in, equal += tie, open += unknown;
          if (!unknown) row.mark(i, in ? kIn : tie ? kTie : kOut);
        }
        __syncwarp();
      }
      if (capped) {  // nothing is above 0: the first zeros are chosen, and the later ones ..
        zeros += __syncthreads_count(lane == 0 && tie);
        sure = __syncthreads_or(unknown) == 0 && sure;
        if (sure && zeros >= want) return {lo, hi, want};  // .. need no look
      }
    }
    above = block_sum<kThreads>(above, sh.sum_a);
    equal = block_sum<kThreads>(equal, sh.sum_a);
    open = block_sum<kThreads>(open, sh.sum_a);
    if (open == 0 && above < want && want <= above + equal) return {lo, hi, want - above};
  }

  // The want-th largest fp64 score, computed anew in each step, then a mark for
  // each candidate. Marks are candidates' from before.
  auto candidate = [&](int32_t i) {
    const uint32_t key = row.key(i);
    return (key >= lo && key <= hi) || key == kIn || key == kTie || key == kOut;
  };
  auto exact = [&](int32_t i) {  // one warp
    uint64_t best = 0;
    pieces(i, [&](int32_t pos, int of) {
      const uint64_t e = exact_key<kTokens>(p, sh, seq, pos, of);
      best = best > e ? best : e;
      return true;
    });
    return best;
  };
  auto each_exact = [&](auto&& f) {
#pragma unroll 1
    for (int32_t i = warp; i < count; i += kWarps) {
      if (!candidate(i)) continue;
      const uint64_t e = exact(i);
      if (lane == 0) f(e);
    }
  };
  uint32_t rank = want;
  const uint64_t edge = kth_largest<kThreads, uint64_t>(sh, uint64_t{0}, ~uint64_t{0}, rank,
                                                        each_exact);
#pragma unroll 1
  for (int32_t i = warp; i < count; i += kWarps) {
    if (!candidate(i)) continue;
    const uint64_t e = exact(i);
    __syncwarp();
    if (lane == 0) row.mark(i, e > edge ? kIn : e == edge ? kTie : kOut);
    __syncwarp();
  }
  __syncthreads();
  return {lo, hi, static_cast<int32_t>(rank)};
}

// The border of the k highest of the `count` keys of a row. `row` gives keys
// by position and their blocks, and takes marks (kIn, kTie, kOut).
template <int kThreads, typename Row>
__device__ __forceinline__ Border choose(const SelectParams& p, SelShared<kThreads>& sh,
                                         const Row& row, const float* scores, int32_t count,
                                         int32_t k, int32_t seq, int32_t seen, float m) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  auto each = [&](auto&& f) {
    for (int32_t i = tid; i < count; i += kThreads) f(row.key(i));
  };
  uint32_t lowest, highest, rank = k;
  key_range(sh, lowest, highest, each);
  const uint32_t tk = kth_largest<kThreads, uint32_t>(sh, lowest, highest, rank, each);
  const float T = unkey32(tk);
  const float eps2 =
      m == 0.f ? 0.f
               : __fadd_ru(__fmul_ru(m, 2.0f * (kDotError + (p.num_heads / 8 + 4) / 16777216.0f)),
                           kTiny);
  // A score of -inf comes from a NaN or a page that does not resolve, not from
  // rounding, unless fp32 overflowed.
  const bool bounded = m < 1e37f;
  if (bounded && (eps2 == 0.f || T == -INFINITY)) return {tk, tk, static_cast<int32_t>(rank)};
  const uint32_t lo = bounded ? key32(__fadd_rd(T, -eps2)) : 1u;
  const uint32_t hi = bounded ? key32(__fadd_ru(T, eps2)) : kTie - 1;

  if (tid == 0) sh.n = 0;
  __syncthreads();
  int in = 0;
  for (int32_t i = tid; i < count; i += kThreads) {
    const uint32_t key = row.key(i);
    if (key > hi) {
      ++in;
    } else if (key >= lo) {
      const uint32_t c = atomicAdd(&sh.n, 1u);
      if (c < SelShared<kThreads>::kCands) sh.cand[c] = i;
    }
  }
  in = block_sum<kThreads>(in, sh.sum_a);
  const int32_t cands = static_cast<int32_t>(sh.n);
  int32_t want = k - in;  // 1 <= want <= cands
  if (cands == want) return {lo, hi, INT32_MAX};  // all of them

  // A warp's piece of a candidate: consecutive positions. None of a granule
  // whose stored score is more than eps2 below the block's can be its highest.
  const int per_piece = min(p.block, kTokens), piece_shift = __ffs(p.block / per_piece) - 1;
  const int granule = min(p.block, kMaxGranule);
  auto piece = [&](int i, int& c, int32_t& pos) {  // how many positions
    // the candidates' first pieces, then their second ones, ..
    const int part = piece_shift == 0 ? 0 : i / cands;
    c = i - part * cands;
    const int off = part * per_piece;
    const int64_t b = row.block(sh.cand[c]), first = b * p.block + off;
    if (first >= seen) return 0;
    pos = static_cast<int32_t>(first);
    if (granule < p.block && bounded &&
        __ldcg(scores + b * (p.block / granule) + off / granule) <
            __fadd_rd(unkey32(row.key(sh.cand[c])), -eps2))
      return 0;
    return min(per_piece, seen - pos);
  };
  if (cands <= SelShared<kThreads>::kCands) {
    for (int i = tid; i < cands; i += kThreads)
      sh.cand_key[i] = 0, sh.cand_lo[i] = sh.cand_hi[i] = 0;
    // Without a positive weight no score is above 0, and a block that has one
    // of 0 is known.
    const bool capped = __syncthreads_or(tid < p.num_heads && sh.w[min(tid, p.num_heads - 1)] > 0.f) == 0;
    auto rescore = [&](auto tokens) {
      constexpr int kTok = decltype(tokens)::value;
#pragma unroll 1
      for (int i = warp; i < cands << piece_shift; i += kWarps) {
        int c;
        int32_t pos;
        const int of = piece(i, c, pos);
        if (of == 0) continue;
        if (capped && __shfl_sync(0xffffffffu, load_volatile(&sh.cand_lo[c]), 0) == key32(0.f))
          continue;
        float low = -INFINITY, high = -INFINITY;
        widen<kTok>(p, sh, seq, pos, of, low, high);
        if (capped) high = fminf(high, 0.f);
        if (lane == 0) {
          atomicMax(&sh.cand_lo[c], key32(low));
          atomicMax(&sh.cand_hi[c], key32(high));
        }
      }
    };
    if (p.block == 1) rescore(Count<1>{}); else rescore(Count<kTokens>{});
    __syncthreads();
    // Known by their intervals: in where fewer than `want` others can be
    // above, out where `want` others are. sh.cand_key: 0 open, 1 in, 2 out.
    int sure = 0;
    for (int i = tid; i < cands; i += kThreads) {
      int can = 0, are = 0;
      for (int j = 0; j < cands; ++j) {
        can += j != i && sh.cand_hi[j] >= sh.cand_lo[i];
        are += sh.cand_lo[j] > sh.cand_hi[i];
      }
      const int state = can < want ? 1 : are >= want ? 2 : 0;
      sh.cand_key[i] = state;
      if (state != 0) row.mark(sh.cand[i], state == 1 ? kIn : kOut);
      sure += state == 1;
    }
    want -= block_sum<kThreads>(sure, sh.sum_a);
    // The best of the others by their fp64 scores, which an interval of one
    // value gives too. sh.cand_hi: 0 known, 1 to be scored, 2 open and exact.
    if (want > 0) {
      for (int i = tid; i < cands; i += kThreads) {
        const uint32_t low = sh.cand_lo[i];
        const bool exact = low == sh.cand_hi[i];
        sh.cand_hi[i] = sh.cand_key[i] != 0 ? 0u : exact ? 2u : 1u;
        sh.cand_key[i] = exact ? key64(static_cast<double>(unkey32(low))) : 0u;
      }
      __syncthreads();
#pragma unroll 1
      for (int i = warp; i < cands << piece_shift; i += kWarps) {
        int c;
        int32_t pos;
        const int of = piece(i, c, pos);
        if (of == 0 || sh.cand_hi[c] != 1) continue;
        const uint64_t key = p.block == 1 ? exact_key<1>(p, sh, seq, pos, 1)
                                          : exact_key<kTokens>(p, sh, seq, pos, of);
        if (lane == 0)
          atomicMax(reinterpret_cast<unsigned long long*>(&sh.cand_key[c]),
                    static_cast<unsigned long long>(key));
      }
      __syncthreads();
      for (int i = tid; i < cands; i += kThreads) {
        if (sh.cand_hi[i] == 0) continue;
        const uint64_t key = sh.cand_key[i];
        const int32_t b = row.block(sh.cand[i]);
        int better = 0;
        for (int j = 0; j < cands; ++j)
          better += sh.cand_hi[j] != 0 &&
                    (sh.cand_key[j] > key || (sh.cand_key[j] == key && row.block(sh.cand[j]) < b));
        row.mark(sh.cand[i], better < want ? kIn : kOut);
      }
    } else {
      for (int i = tid; i < cands; i += kThreads)
        if (sh.cand_key[i] == 0) row.mark(sh.cand[i], kOut);
    }
    __syncthreads();
    return {lo, hi, 0};
  }

  return choose_unlisted<kThreads>(p, sh, row, count, want, seq, seen, lo, hi);
}

// ------------------------------------------------------------------- rows
// A row's scores in memory: a block's is the highest of its `per` stored ones.
// A mark is a NaN's word in the place of a block's first score. It is loaded as
// a word: a float on its way through the compiler need not keep a NaN's payload,
// and a float load here was seen to lose it.
struct MemoryRow {
  float* scores;
  int32_t b0, per, granules;
  __device__ __forceinline__ int32_t block(int32_t i) const { return b0 + i; }
  __device__ __forceinline__ uint32_t* word(int64_t at) const {
    return reinterpret_cast<uint32_t*>(scores) + at;
  }
  __device__ __forceinline__ uint32_t key(int32_t i) const {
    const int64_t at = static_cast<int64_t>(b0 + i) * per;
    const uint32_t u = __ldcg(word(at));
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return u >> 31 ? ~u : u | 0x80000000u;  // a mark
    float a = __uint_as_float(u);
    for (int g = 1; g < per; ++g)
      if (at + g < granules) a = fmaxf(a, __ldcg(scores + at + g));
    return key32(a);
  }
  __device__ __forceinline__ void mark(int32_t i, uint32_t m) const {
    *word(static_cast<int64_t>(b0 + i) * per) = m == kOut ? 0xFFFFFFFFu : m & 0x7FFFFFFFu;
  }
};
struct DenseRow {  // shared memory, all blocks from b0 on
  uint32_t* keys;
  int32_t b0;
  __device__ __forceinline__ int32_t block(int32_t i) const { return b0 + i; }
  __device__ __forceinline__ uint32_t key(int32_t i) const { return keys[i]; }
  __device__ __forceinline__ void mark(int32_t i, uint32_t m) const { keys[i] = m; }
};
struct ListRow {  // shared memory, some blocks in any order
  uint32_t* keys;
  int32_t* blocks;
  __device__ __forceinline__ int32_t block(int32_t i) const { return blocks[i]; }
  __device__ __forceinline__ uint32_t key(int32_t i) const { return keys[i]; }
  __device__ __forceinline__ void mark(int32_t i, uint32_t m) const { keys[i] = m; }
};

// Output row of a query token: the first positions of its num_select blocks are
// written in order, the others follow from them.
template <int kThreads>
__device__ __forceinline__ void expand_blocks(const SelectParams& p, int32_t* out, int64_t width,
                                              int32_t seen) {
  if (p.block == 1) return;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < width; i += kThreads) {
    const int off = static_cast<int>(i) & (p.block - 1);
    if (off == 0) continue;
    const int32_t pos = __ldcg(out + (i - off)) + off;
    out[i] = pos < seen ? pos : -1;
  }
}

// The first positions of the chosen blocks in order, `row` holding the blocks
// from p.sink on: num_select ones, as there are more blocks than that. A warp has
// consecutive blocks: it counts, learns what comes before it, and writes.
template <int kThreads, typename Row>
__device__ __forceinline__ void emit_row(const SelectParams& p, SelShared<kThreads>& sh,
                                         const Row& row, const Border& border, int32_t blocks,
                                         int32_t* out) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t share = ((blocks + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int32_t from = min(warp * share, blocks), to = min(from + share, blocks);
  auto state = [&](int32_t b, bool& tie) {
    tie = false;
    if (b >= to) return false;
    if (b < p.sink || b >= blocks - p.recent) return true;
    const uint32_t key = row.key(b - p.sink);
    tie = key == kTie || (key >= border.lo && key <= border.hi);
    return key > border.hi && !tie;
  };
  int sure = 0, ties = 0;
  for (int32_t b0 = from; b0 < to; b0 += 32) {
    bool tie;
    const bool in = state(b0 + lane, tie);
    sure += __popc(__ballot_sync(0xffffffffu, in));
    ties += __popc(__ballot_sync(0xffffffffu, tie));
  }
  int total;
  int32_t tie_at = 0;
  if (border.ties > 0) {
    tie_at = block_before<kThreads>(lane == 0 ? ties : 0, sh.sum_a, total);
    tie_at = __shfl_sync(0xffffffffu, tie_at, 0);
  }
  const int taken = max(0, min(ties, border.ties - tie_at));
  int32_t at = block_before<kThreads>(lane == 0 ? sure + taken : 0, sh.sum_b, total);
  at = __shfl_sync(0xffffffffu, at, 0);
  for (int32_t b0 = from; b0 < to; b0 += 32) {
    bool tie;
    bool in = state(b0 + lane, tie);
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    in = in || (tie && tie_at + __popc(tied & ((1u << lane) - 1)) < border.ties);
    tie_at += __popc(tied);
    const uint32_t chosen = __ballot_sync(0xffffffffu, in);
    const int32_t slot = at + __popc(chosen & ((1u << lane) - 1));
    if (in && slot < p.num_select)
      out[static_cast<int64_t>(slot) * p.block] = (b0 + lane) * p.block;
    at += __popc(chosen);
  }
}

__device__ __forceinline__ uint32_t sel_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t sel_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void sel_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t in_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

// The long row: this CTA's share from .. to - 1 of the keys that are at least
// `floor`, into the list of `cap` entries; returns how many there are (some
// may not have fitted). `from` is a multiple of 4.
template <int kThreads>
__device__ __forceinline__ int32_t collect(SelShared<kThreads>& sh, const MemoryRow& row,
                                           int32_t from, int32_t to, uint32_t floor,
                                           uint32_t* keys, int32_t* blocks, int32_t cap) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) sh.n = 0;
  __syncthreads();
  constexpr int kQuads = 2;  // 8 keys of a thread at a time
  // one stored score a block, 16-byte aligned: four at once
  const bool vec = row.per == 1 && row.b0 % 4 == 0;
  for (int32_t i0 = from; i0 < to; i0 += kThreads * 4 * kQuads) {
    uint32_t key[4 * kQuads];
    uint32_t hits = 0;
    if (vec && i0 + kThreads * 4 * kQuads <= to) {
      float4 v[kQuads];
#pragma unroll
      for (int u = 0; u < kQuads; ++u)
        v[u] = __ldcg(reinterpret_cast<const float4*>(row.scores + row.b0 + i0) + u * kThreads +
                      threadIdx.x);
#pragma unroll
      for (int u = 0; u < kQuads; ++u) {
        key[4 * u] = key32(v[u].x), key[4 * u + 1] = key32(v[u].y);
        key[4 * u + 2] = key32(v[u].z), key[4 * u + 3] = key32(v[u].w);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4 * kQuads; ++u) {
        const int64_t i = static_cast<int64_t>(i0) + (u >> 2) * kThreads * 4 + threadIdx.x * 4 + (u & 3);
        key[u] = i < to ? row.key(static_cast<int32_t>(i)) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < 4 * kQuads; ++u) hits |= (key[u] >= floor ? 1u : 0u) << u;
    const int mine = __popc(hits);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    uint32_t at = 0;
    if (lane == 31 && upto > 0) at = atomicAdd(&sh.n, static_cast<uint32_t>(upto));
    at = __shfl_sync(0xffffffffu, at, 31) + upto - mine;
    if (hits != 0) {
#pragma unroll
      for (int u = 0; u < 4 * kQuads; ++u) {
        if ((hits >> u & 1u) == 0) continue;
        if (at < static_cast<uint32_t>(cap)) {
          keys[at] = key[u];
          blocks[at] = row.block(i0 + (u >> 2) * kThreads * 4 + static_cast<int32_t>(threadIdx.x) * 4 +
                                 (u & 3));
        }
        ++at;
      }
    }
  }
  __syncthreads();
  return static_cast<int32_t>(sh.n);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    select_kernel(const SelectParams p, const SelectConfig cfg) {
  using Shared = SelShared<kThreads>;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(raw + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ctas = sel_ctas(), rank = sel_rank();
  const int32_t t = blockIdx.x / ctas;
  const int64_t width = static_cast<int64_t>(p.num_select) * p.block;
  int32_t* out = p.topk_idx + t * width;
  const int32_t seq = __ldg(p.q_seq + t);
  const int32_t seen = visible_positions(p, seq, __ldg(p.q_pos + t));
  const int32_t blocks = (seen + (p.block - 1)) >> (__ffs(p.block) - 1);
  const bool all = seen <= p.take_all;

  // The heads as integers, and their part of the error bound: nothing that
  // the score kernel writes.
  float m = 0.f;
  if (!all) {
    for (int g = tid; g < p.num_heads * kIndexScales; g += kThreads) {
      const uint8_t* src =
          p.q_index + (static_cast<int64_t>(t) * p.num_heads * kIndexScales + g) * (2 * kGroup);
      const uint4 a = ld_nc_v4(src), b = ld_nc_v4(src + 16);
      const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const int j = g / kIndexScales, part = g % kIndexScales;
      uint32_t c[2];
      float s;
      sh.q_scale[part][j] = static_cast<uint16_t>(scale_parts(quantize_group(v, c[0], c[1], s)));
      int mag = 0;
      uint32_t e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[i] = expand_codes(c[i >> 1] >> (16 * (i & 1)));
        mag = __dp4a(static_cast<int>(__vabs4(e[i])), 0x01010101, mag);
      }
      sh.q_codes[part][j] = make_uint4(e[0], e[1], e[2], e[3]);
      const float w = __ldg(p.weights + static_cast<int64_t>(t) * p.num_heads + j);
      if (part == 0) sh.w[j] = w;
      m = fmaf(fabsf(w), 0.5f * mag * s, m);
      if (mag > 0 && w != 0.f) m += kTiny;  // never 0 by underflow
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m += __shfl_xor_sync(0xffffffffu, m, d);
    if (lane == 0) sh.red[warp] = m;
  }
  if (tid == 0) sh.failed = 0;
  __syncthreads();
  cudaGridDependencySynchronize();  // the scores are there
  for (int i = tid; i < p.score_ctas; i += kThreads)
    if (__ldcg(p.status + i) != 0) sh.failed = 1;
  __syncthreads();
  if (sh.failed || all) {
    if (rank == 0)
      for (int64_t i = tid; i < width; i += kThreads)
        out[i] = sh.failed ? -2 : i < seen ? static_cast<int32_t>(i) : -1;
    return;
  }

  // The forced blocks are at both ends: k of the n between them are chosen.
  const int granule = min(p.block, kMaxGranule);
  const MemoryRow row = {p.scores + t * p.score_stride, p.sink, p.block / granule,
                         (seen + granule - 1) / granule};
  const int32_t n = blocks - p.sink - p.recent;
  const int32_t k = p.num_select - p.sink - p.recent;
  // A cluster is launched for what the table can hold; a row without a long
  // sweep is one CTA's.
  if (rank > 0 && (k == 0 || n <= cfg.room)) return;
  if (k == 0) {
    emit_row<kThreads>(p, sh, row, Border{kTie, kTie, 0}, blocks, out);
    expand_blocks<kThreads>(p, out, width, seen);
    return;
  }
  {
    int32_t lead = t;  // first token of t's run
    while (lead % p.group != 0 && __ldg(p.q_seq + lead - 1) == seq) --lead;
    uint32_t top = 0;
    const int32_t tiles = (seen + kScoreTile - 1) / kScoreTile;
    for (int32_t i = tid; i < tiles; i += kThreads)
      top = __vmaxu4(top, __ldcg(p.smax + lead * p.tiles + i));
    top = __vmaxu4(top, top >> 16);
    top = __reduce_max_sync(0xffffffffu, __vmaxu4(top, top >> 8) & 0xFFu);
    if (lane == 0) sh.redu[warp] = top;
    __syncthreads();
    m = lane < kWarps ? sh.red[lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m += __shfl_xor_sync(0xffffffffu, m, d);
    top = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.redu[lane] : 0u);
    // a little more than 6: the sum's own rounding
    m = __fmul_ru(m, 6.001f * scale_value(top));
    __syncthreads();
  }

  if (n <= cfg.room) {
    const DenseRow dense = {keys, p.sink};
    for (int32_t i = tid; i < n; i += kThreads) keys[i] = row.key(i);
    __syncthreads();
    const Border border = choose<kThreads>(p, sh, dense, row.scores, n, k, seq, seen, m);
    emit_row<kThreads>(p, sh, dense, border, blocks, out);
    expand_blocks<kThreads>(p, out, width, seen);
    return;
  }

  if constexpr (kThreads > 256) {
    // A threshold that about k + 4 sqrt(k) scores pass, by a sample's share.
    const int32_t cap = cfg.room / 2;
    int32_t* list_blocks = reinterpret_cast<int32_t*>(keys + cap);
    const float share = static_cast<float>(k) * kSample / static_cast<float>(n);
    uint32_t from_top = static_cast<uint32_t>(share + 4.f * sqrtf(share) + 8.f);
    const float expect = static_cast<float>(from_top) * n / kSample;
    bool listed = expect < 0.9f * cap && (blocks + 127) / 128 * 4 <= cfg.room;
    if (listed) {
      for (int32_t i = tid; i < kSample; i += kThreads)
        keys[i] = row.key(static_cast<int32_t>(static_cast<int64_t>(i) * n / kSample));
      __syncthreads();
      auto each = [&](auto&& f) {
        for (int32_t i = tid; i < kSample; i += kThreads) f(keys[i]);
      };
      uint32_t lowest, highest;
      key_range(sh, lowest, highest, each);
      // Two levels leave the threshold within 2^-14 or so of its value; one
      // would not, as keys are spaced like exponents and scores of both signs
      // spread over nearly all of them.
      const uint32_t floor =
          kth_largest<kThreads, uint32_t, 2>(sh, lowest, highest, from_top, each);
      const int32_t per = ((n + static_cast<int32_t>(ctas) - 1) / static_cast<int32_t>(ctas) + 3) / 4 * 4;
      const int32_t from = min(static_cast<int32_t>(rank) * per, n);
      const int32_t mine =
          collect<kThreads>(sh, row, from, min(from + per, n), floor, keys, list_blocks, cap);
      int32_t count = mine;
      if (ctas > 1) {  // the lists go behind one another into rank 0's
        if (tid == 0) sh.sum_a[0] = mine;
        sel_cluster_sync();
        int32_t before = 0;
        count = 0;
        for (uint32_t r = 0; r < ctas; ++r) {
          int32_t c;
          asm volatile("ld.shared::cluster.s32 %0, [%1];"
                       : "=r"(c)
                       : "r"(in_rank(smem_u32(&sh.sum_a[0]), r))
                       : "memory");
          if (r < rank) before += c;
          count += c;
        }
        if (rank > 0 && count <= cap) {
          const uint32_t to_keys = in_rank(smem_u32(keys), 0);
          const uint32_t to_blocks = in_rank(smem_u32(list_blocks), 0);
          for (int32_t i = tid; i < mine; i += kThreads) {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to_keys + 4u * (before + i)),
                         "r"(keys[i])
                         : "memory");
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to_blocks + 4u * (before + i)),
                         "r"(list_blocks[i])
                         : "memory");
          }
        }
        sel_cluster_sync();
      }
      if (rank > 0) return;
      listed = count <= cap && count >= k;
      if (listed) {
        const ListRow list = {keys, list_blocks};
        const Border border = choose<kThreads>(p, sh, list, row.scores, count, k, seq, seen, m);
        // What lies at the border has to have passed the threshold; the first
        // ones of a tie cannot be told in a list.
        listed = border.lo >= floor && (border.ties == 0 || border.ties == INT32_MAX);
        if (listed) {
          // the chosen ones as bits, in the list's place
          constexpr int kPer = (kThreads == 1024 ? kWideRoom : kRoom) / 2 / kThreads;
          int32_t mine_in[kPer];
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int32_t i = u * kThreads + tid;
            mine_in[u] = -1;
            if (u * kThreads >= count) continue;
            if (i < count) {
              const uint32_t key = keys[i];
              if (key > border.hi || (border.ties > 0 && key >= border.lo))
                mine_in[u] = list_blocks[i];
            }
          }
          __syncthreads();
          uint4* bits4 = reinterpret_cast<uint4*>(keys);
          const int32_t quads = (blocks + 127) / 128;
          for (int32_t i = tid; i < quads; i += kThreads) bits4[i] = make_uint4(0, 0, 0, 0);
          __syncthreads();
#pragma unroll
          for (int u = 0; u < kPer; ++u)
            if (u * kThreads < count && mine_in[u] >= 0) atomicOr(&keys[mine_in[u] >> 5], 1u << (mine_in[u] & 31));
          for (int32_t i = tid; i < p.sink + p.recent; i += kThreads) {
            const int32_t b = i < p.sink ? i : blocks - 1 - (i - p.sink);
            atomicOr(&keys[b >> 5], 1u << (b & 31));
          }
          __syncthreads();
          // a warp's share of the bits, 32 lanes x 128 at a time
          const int32_t share4 = ((quads + kWarps - 1) / kWarps + 31) / 32 * 32;
          const int32_t w0 = min(warp * share4, quads), w1 = min(w0 + share4, quads);
          int bits = 0;
          for (int32_t i = w0 + lane; i < w1; i += 32) {
            const uint4 v = bits4[i];
            bits += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
          }
          bits = __reduce_add_sync(0xffffffffu, bits);
          int total;
          int at = block_before<kThreads>(lane == 0 ? bits : 0, sh.sum_a, total);
          at = __shfl_sync(0xffffffffu, at, 0);
          for (int32_t i0 = w0; i0 < w1; i0 += 32) {
            const uint4 v = i0 + lane < w1 ? bits4[i0 + lane] : make_uint4(0, 0, 0, 0);
            const int mine_bits = __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
            int upto = mine_bits;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const int o = __shfl_up_sync(0xffffffffu, upto, d);
              if (lane >= d) upto += o;
            }
            int64_t slot = at + upto - mine_bits;
            at += __shfl_sync(0xffffffffu, upto, 31);
            const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
              for (uint32_t left = word[u]; left != 0 && slot < p.num_select; left &= left - 1)
                out[slot++ * p.block] = (((i0 + lane) * 4 + u) * 32 + __ffs(left) - 1) * p.block;
          }
          expand_blocks<kThreads>(p, out, width, seen);
          return;
        }
      }
      __syncthreads();
    }
    if (rank > 0) return;
    const Border border = choose<kThreads>(p, sh, row, row.scores, n, k, seq, seen, m);
    emit_row<kThreads>(p, sh, row, border, blocks, out);
    expand_blocks<kThreads>(p, out, width, seen);
  }
}

// Largest room that launch_select<kThreads> is called with or takes.
constexpr int kSmallRoom = 4096;
constexpr int most_room(int threads) {
  return threads == 256 ? kSmallRoom : threads == 512 ? kRoom : kWideRoom;
}

template <int kThreads>
int32_t launch_select(const SelectParams& p, int32_t most_blocks, int num_sms,
                      cudaStream_t stream) {
  SelectConfig cfg;
  cfg.room = most_blocks <= kRoom ? most_blocks : most_blocks <= 32 * kRoom ? kRoom : kWideRoom;
  // A cluster per query token where the rows are long and the device is not
  // full: one row of a million scores 59 us with it, 145 without; 66 rows of
  // 146000 54 and 61.
  int ctas = 1;
  if (most_blocks > kWideRoom)
    while (ctas < kMaxCluster && p.num_q * ctas * 2 <= num_sms) ctas *= 2;
  const size_t smem = sizeof(SelShared<kThreads>) + 4 * static_cast<size_t>(cfg.room);
  // The limit is the process's: calls of other threads rely on it, so that it is
  // the same one in every call.
  constexpr size_t kMost = sizeof(SelShared<kThreads>) + 4 * static_cast<size_t>(most_room(kThreads));
  static_assert(kMost <= kMaxSharedBytes, "shared memory");
  if (smem > kMost ||
      cudaFuncSetAttribute(select_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kMost)) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  cudaLaunchConfig_t launch = {};
  launch.gridDim = dim3(static_cast<unsigned>(p.num_q) * ctas);
  launch.blockDim = dim3(kThreads);
  launch.dynamicSmemBytes = smem;
  launch.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // starts as the score kernel's CTAs end; it waits for the scores itself
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  launch.attrs = attr;
  launch.numAttrs = 2;
  if (cudaLaunchKernelEx(&launch, select_kernel<kThreads>, p, cfg) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  return NVFP4_MLA_OK;
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
  w.per_q = static_cast<size_t>(w.score_stride + w.tiles) * 4 + query_image_bytes(num_heads);
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
    p.room = max_blocks_per_seq * page_size;
    p.take_all = num_select * select_block;
    p.topk_idx = topk_idx + static_cast<int64_t>(q0) * num_select * select_block;
    p.images = static_cast<uint8_t*>(workspace);
    p.scores = reinterpret_cast<float*>(p.images + query_image_bytes(num_heads) * w.chunk);
    p.score_stride = w.score_stride;
    p.smax = reinterpret_cast<uint32_t*>(p.scores + w.score_stride * w.chunk);
    p.tiles = w.tiles;
    p.status = reinterpret_cast<uint32_t*>(p.smax + w.tiles * w.chunk);
    p.wait_cycles = decode_wait_cycles();
    if (int32_t st = launch_scores(p, sms, s)) return st;
    const int32_t most_blocks = static_cast<int32_t>(
        (static_cast<int64_t>(max_blocks_per_seq) * page_size + select_block - 1) / select_block);
    // Where there are more query tokens than SMs, smaller CTAs share an SM: one's
    // barriers and loads pass while another works. 2048 rows of 1024 blocks: 80 us
    // with 256 threads, 105 with 512, 172 with 1024. 480 rows of 65536 blocks: 193
    // us with 512, 224 with 1024 (most of both beside the end of the scoring, which
    // was longer then). 66
    // rows of 146000: 76 us with 512, 54 with 1024.
    const bool many = p.num_q > 2 * sms;
    const int32_t st = many && most_blocks <= kSmallRoom   ? launch_select<256>(p, most_blocks, sms, s)
                       : many && most_blocks <= 32 * kRoom ? launch_select<512>(p, most_blocks, sms, s)
                                                           : launch_select<1024>(p, most_blocks, sms, s);
    if (st != NVFP4_MLA_OK) return st;
  }
  return NVFP4_MLA_OK;
}
