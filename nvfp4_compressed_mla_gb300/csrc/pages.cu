// pages.cu -- pages that several sequences share: forking, releasing, compacting and copying.
//
// page_shares[p] counts the holders of page p beyond the first, so that a free
// page and a page with one holder both have 0 and nvfp4_mla_plan_step, which
// hands out pages that have one, needs no knowledge of it. A fork shares whole
// pages only and copies a partly filled last page, so no sequence ever appends
// to a page that another one reads.
//
// All four work on metadata of a few kilobytes to a few megabytes and are bound
// by latency (dependent loads, launches, barriers), but for the copy of pages,
// which is bound by HBM: it reads and writes each page once. Measured, device time of
// each kernel alone (a launch's 2 us and cold loads included):
//   fork      32 forks of up to 62 pages     plan 6.3 us, share 4.9
//             960 forks of up to 125 pages   plan 7.9 us, share 6.0; together, in a graph, 7
//   release   128 sequences of up to 97 pages  15.2 us; 1000 of up to 506 pages 23.4 us
//   compact   16 sequences, 888 pages        4.7 + 4.8 + 8.3 + 4.5 us (clear, mark, rank, table)
//             100 sequences, 23081 pages     5.0 + 6.0 + 11.8 + 4.8 us
//   copy      5510 pages of 22.5 KB          38.4 us, 6.5 TB/s (a plain copy of the device: 6.8)
// A fork in one launch of a cluster, plan and shares one behind the other, takes as long
// on the device for up to 32 forks (4.8 us in a graph) and longer from 64 on (5.5 for
// 4.8), so that there is no such variant.
#include <atomic>

#include "plan_common.cuh"

namespace nvfp4_mla {
namespace {

constexpr int kRowThreads = 256;      // CTAs that walk rows of a table
constexpr int kRowChunk = 1024;       // entries of a row that such a CTA takes at a time
constexpr int kCopyVecs = 4;          // 16-byte vectors that a copying thread has under way

// ------------------------------------------------------------------------- fork
struct ForkParams {
  const int32_t* src_seqs;
  const int32_t* dst_seqs;
  const int32_t* fork_lens;
  int32_t num_forks;
  const int32_t* seq_lens;
  int32_t num_seqs;
  int32_t* block_table;
  int32_t max_blocks;
  PageSize page;
  const int32_t* page_shares;
  int32_t num_blocks;
  const int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int32_t* seq_lens_out;
  int32_t* page_shares_out;
  int32_t* free_count_out;
  int32_t* shared_blocks;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* refused_count;
};

__device__ __forceinline__ void copy_ints(const int32_t* __restrict__ from, int32_t* __restrict__ to,
                                          int64_t n, int64_t first, int64_t stride) {
  for (int64_t i = first; i < n; i += 4 * stride) {
    int32_t v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * stride < n) v[u] = __ldg(from + i + u * stride);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * stride < n) to[i + u * stride] = v[u];
  }
}

// CTA 0 decides which forks are served (one prefix sum over the fresh pages
// that they need) and writes all but the shared entries; the other CTAs copy
// the counts of holders where those go to another buffer.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams p) {
  extern __shared__ int32_t claim[];  // [num_seqs] first fork that names the sequence as its dst
  __shared__ int64_t sums[32];
  const int tid = threadIdx.x;
  cudaTriggerProgrammaticLaunchCompletion();
  if (blockIdx.x > 0) {
    copy_ints(p.page_shares, p.page_shares_out, p.num_blocks,
              static_cast<int64_t>(blockIdx.x - 1) * kPlanThreads + tid,
              static_cast<int64_t>(gridDim.x - 1) * kPlanThreads);
    return;
  }
  // an ordinary load: the count may be replaced below
  const int32_t free_now = min(max(*p.free_count, 0), p.free_capacity);
  int32_t src, dst, len;
  auto load = [&](int i) {
    const bool here = i < p.num_forks;
    src = here ? __ldg(p.src_seqs + i) : -1;
    dst = here ? __ldg(p.dst_seqs + i) : -1;
    len = here ? __ldg(p.fork_lens + i) : 0;
  };
  load(tid);  // one round's forks stay in registers
  const bool one = p.num_forks <= kPlanThreads;
  for (int s = tid; s < p.num_seqs; s += kPlanThreads) {
    claim[s] = p.num_forks;
    if (p.seq_lens_out != p.seq_lens) p.seq_lens_out[s] = p.seq_lens[s];
  }
  __syncthreads();
  for (int i = tid; i < p.num_forks; i += kPlanThreads) {
    if (!one) load(i);
    if (src != -1 && dst >= 0 && dst < p.num_seqs) atomicMin(claim + dst, i);
  }
  __syncthreads();
  const int64_t room = static_cast<int64_t>(p.max_blocks) * p.page.size;
  int64_t asked = 0;
  int refused = 0;
  for (int i0 = 0; i0 < p.num_forks; i0 += kPlanThreads) {
    const int i = i0 + tid;
    if (!one) load(i);
    bool ok = src >= 0 && src < p.num_seqs && dst >= 0 && dst < p.num_seqs && len >= 0 &&
              len <= room && claim[min(max(dst, 0), p.num_seqs - 1)] == i;
    // ordinary loads: the lengths may be replaced below
    ok = ok && len <= p.seq_lens[src] && p.seq_lens[dst] == 0;
    const int32_t full = ok ? p.page.block(len) : 0;
    const bool need = ok && len != full * p.page.size;
    const int64_t rank = block_scan(need ? 1 : 0, asked, sums);
    ok = ok && (!need || rank <= free_now);
    int32_t from = -1, to = -1;
    if (ok && need) {
      to = __ldg(p.free_pages + (free_now - rank));
      from = p.block_table[static_cast<int64_t>(src) * p.max_blocks + full];
      p.block_table[static_cast<int64_t>(dst) * p.max_blocks + full] = to;
    }
    if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) from = to = -1;
    if (i < p.num_forks) {
      p.shared_blocks[i] = ok ? full : -1;
      p.copy_src[i] = from;
      p.copy_dst[i] = to;
      if (ok && one) p.seq_lens_out[dst] = len;  // every length was read before the sum
      if (!ok && src != -1) ++refused;
    }
  }
  // the forks up to the first one without a page have one each
  if (tid == 0) *p.free_count_out = free_now - static_cast<int32_t>(min(asked, static_cast<int64_t>(free_now)));
  if (p.refused_count != nullptr && refused > 0) atomicAdd(p.refused_count, refused);
  if (one) return;
  __syncthreads();  // every length has been read
  for (int i = tid; i < p.num_forks; i += kPlanThreads)  // a thread's own results
    if (p.shared_blocks[i] >= 0) p.seq_lens_out[__ldg(p.dst_seqs + i)] = __ldg(p.fork_lens + i);
}

// The shared entries, 1024 of a fork at a time, and their pages' holders.
__global__ void __launch_bounds__(kRowThreads) fork_share_kernel(const ForkParams p, int32_t chunks) {
  cudaGridDependencySynchronize();
  const int64_t units = static_cast<int64_t>(p.num_forks) * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int32_t i = static_cast<int32_t>(u / chunks);
    const int32_t b0 = static_cast<int32_t>(u - static_cast<int64_t>(i) * chunks) * kRowChunk;
    const int32_t full = __ldcg(p.shared_blocks + i);
    if (full <= b0) continue;
    const int32_t* from = p.block_table + static_cast<int64_t>(__ldg(p.src_seqs + i)) * p.max_blocks;
    int32_t* to = p.block_table + static_cast<int64_t>(__ldg(p.dst_seqs + i)) * p.max_blocks;
    int32_t page[kRowChunk / kRowThreads];
#pragma unroll
    for (int k = 0; k < kRowChunk / kRowThreads; ++k) {
      const int32_t b = b0 + k * kRowThreads + threadIdx.x;
      page[k] = b < full ? from[b] : -1;
    }
#pragma unroll
    for (int k = 0; k < kRowChunk / kRowThreads; ++k) {
      const int32_t b = b0 + k * kRowThreads + threadIdx.x;
      if (b < full) to[b] = page[k];
      if (page[k] >= 0 && page[k] < p.num_blocks) atomicAdd(p.page_shares_out + page[k], 1);
    }
  }
}

// ---------------------------------------------------------------------- release
struct ReleaseParams {
  const int32_t* keep_lens;
  const int32_t* seq_lens;
  int32_t num_seqs;
  const int32_t* block_table;
  int32_t max_blocks;
  PageSize page;
  const int32_t* page_shares;
  int32_t num_blocks;
  int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int32_t* seq_lens_out;
  int32_t* page_shares_out;
  int32_t* free_count_out;
  int32_t* dropped_count;
  int32_t* refused_count;
};

constexpr int kReleaseUnits = 4096;  // beside one a sequence
constexpr int kReleaseFlight = 8;    // entries of a lane under way
constexpr int kReleaseChunk = 32 * kReleaseFlight;
constexpr int kReleaseMark = 1 << 20;
constexpr size_t kReleaseBytes = 12;  // of shared memory a sequence, beside the units' 4 each
static_assert(kReleaseBytes * NVFP4_MLA_MAX_PLAN_SEQS + 4 * kReleaseUnits + 512 <= kMaxSharedBytes,
              "shared memory");

// One cluster. The released entries are cut into units of (at least) 256, at
// most kReleaseUnits and one a sequence, which the warps take in turn:
//   1. every entry takes one off its page's count; a page whose count falls
//      below 0 has lost its last holder;
//   2. the first sequence that dropped such a page marks it with its number
//      (the lowest, by an atomic minimum below all counts): that entry is the
//      one that returns the page, whatever the order of the atomics was;
//   3. the units' returned pages are counted, summed up and pushed.
__global__ void __launch_bounds__(kPlanThreads) release_kernel(const ReleaseParams p) {
  extern __shared__ int32_t dyn[];
  int32_t* begin = dyn;                  // [num_seqs] first released block
  int32_t* unit_end = dyn + p.num_seqs;  // [num_seqs] entries, then units up to and with sequence s
  int32_t* counts = unit_end + p.num_seqs;  // [num_seqs + kReleaseUnits] pages of a unit, then sums
  __shared__ int64_t sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cta_rank(), ctas = cluster_size();
  const int32_t free_now = min(max(*p.free_count, 0), p.free_capacity);

  int64_t entries = 0;
  int refused = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int32_t b0 = 0, b1 = 0;
    bool cut = false;
    if (s < p.num_seqs) {
      const int32_t len = p.seq_lens[s], keep = __ldg(p.keep_lens + s);
      cut = keep >= 0 && keep < len;
      if (cut) {
        const int32_t inner = p.page.block(keep);
        if (keep != inner * p.page.size && inner < p.max_blocks) {
          const int32_t page = __ldg(p.block_table + static_cast<int64_t>(s) * p.max_blocks + inner);
          // an ordinary load: the counts may be replaced behind the barrier
          if (page >= 0 && page < p.num_blocks && p.page_shares[page] > 0) {
            cut = false;
            ++refused;
          }
        }
        if (cut) {
          b0 = p.page.blocks(keep);
          b1 = max(min(p.page.blocks(len), p.max_blocks), b0);
        }
      }
      begin[s] = cut ? b0 : -1;
      unit_end[s] = b1 - b0;
    }
    block_scan(b1 - b0, entries, sums);
  }
  const int64_t chunk =
      max((entries + kReleaseUnits - 1) / kReleaseUnits + kReleaseChunk - 1, int64_t{kReleaseChunk}) /
      kReleaseChunk * kReleaseChunk;
  int64_t units_so_far = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const int64_t to = block_scan(s < p.num_seqs ? (unit_end[s] + chunk - 1) / chunk : 0, units_so_far, sums);
    if (s < p.num_seqs) unit_end[s] = static_cast<int32_t>(to);
  }
  const int units = static_cast<int>(units_so_far);
  if (p.page_shares_out != p.page_shares)
    copy_ints(p.page_shares, p.page_shares_out, p.num_blocks,
              static_cast<int64_t>(rank) * kPlanThreads + tid, static_cast<int64_t>(ctas) * kPlanThreads);
  if (rank == 0 && p.refused_count != nullptr && refused > 0) atomicAdd(p.refused_count, refused);
  __syncthreads();  // the units are in shared memory

  const int first_unit = static_cast<int>(rank) * kPlanWarps + warp;
  const int stride = static_cast<int>(ctas) * kPlanWarps;
  // the sequence of a unit, its next block and the block behind its last
  auto locate = [&](int u, int& s, int64_t& b, int64_t& end) {
    int lo = 0, hi = p.num_seqs;  // the first sequence whose units end behind u
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (unit_end[mid] <= u) lo = mid + 1;
      else hi = mid;
    }
    s = lo;
    b = begin[s] + (u - (s > 0 ? unit_end[s - 1] : 0)) * chunk;
    end = min(b + chunk, static_cast<int64_t>(min(p.page.blocks(p.seq_lens[s]), p.max_blocks)));
  };
  auto load = [&](int s, int64_t b, int64_t end, int32_t (&page)[kReleaseFlight]) {
    const int32_t* row = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
#pragma unroll
    for (int k = 0; k < kReleaseFlight; ++k) {
      const int64_t at = b + 32 * k + lane;
      page[k] = at < end ? __ldg(row + at) : -1;
      if (page[k] >= p.num_blocks) page[k] = -1;
    }
  };
  // The warp's first two units stay in registers through the passes, if they are of
  // one round each.
  constexpr int kKept = 2;
  int kept_seq[kKept];
  int32_t kept[kKept][kReleaseFlight];
  const bool keeps = chunk == kReleaseChunk;
  if (keeps) {
#pragma unroll
    for (int x = 0; x < kKept; ++x) {
      const int u = first_unit + x * stride;
      int64_t b = 0, end = 0;
      kept_seq[x] = 0;
      if (u < units) locate(u, kept_seq[x], b, end);
      load(kept_seq[x], b, end, kept[x]);
    }
  }
  // which of the kept entries return their page: a bit each, known behind the third pass
  uint32_t ours[kKept] = {};
  // start(u), f(s, pages of 8 x 32 entries (-1: none), their place in `ours` or null) for each
  // round of the warp's units, and stop(u)
  auto walk = [&](auto&& start, auto&& f, auto&& stop) {
    if (keeps) {
#pragma unroll
      for (int x = 0; x < kKept; ++x) {
        const int u = first_unit + x * stride;
        if (u < units) {
          start(u);
          f(kept_seq[x], kept[x], ours + x);
          stop(u);
        }
      }
    }
    for (int u = first_unit + (keeps ? kKept * stride : 0); u < units; u += stride) {
      int s;
      int64_t b, end;
      locate(u, s, b, end);
      start(u);
      for (; b < end; b += kReleaseChunk) {
        int32_t page[kReleaseFlight];
        load(s, b, end, page);
        f(s, page, static_cast<uint32_t*>(nullptr));
      }
      stop(u);
    }
  };
  auto nothing = [](int) {};
  auto held_by = [&](const int32_t(&page)[kReleaseFlight], int32_t (&held)[kReleaseFlight]) {
#pragma unroll
    for (int k = 0; k < kReleaseFlight; ++k)
      held[k] = page[k] >= 0 ? __ldcg(p.page_shares_out + page[k]) : 0;
  };

  cluster_barrier();  // the counts may change now
  walk(nothing, [&](int, const int32_t(&page)[kReleaseFlight], uint32_t*) {
#pragma unroll
    for (int k = 0; k < kReleaseFlight; ++k)
      if (page[k] >= 0) atomicAdd(p.page_shares_out + page[k], -1);
  }, nothing);
  cluster_barrier();
  walk(nothing, [&](int s, const int32_t(&page)[kReleaseFlight], uint32_t*) {
    int32_t held[kReleaseFlight];
    held_by(page, held);
#pragma unroll
    for (int k = 0; k < kReleaseFlight; ++k)
      if (held[k] < 0) atomicMin(p.page_shares_out + page[k], s - kReleaseMark);
  }, nothing);
  cluster_barrier();
  const uint32_t counts_addr = smem_u32(counts);
  int n = 0;
  walk([&](int) { n = 0; },
       [&](int s, const int32_t(&page)[kReleaseFlight], uint32_t* out) {
         int32_t held[kReleaseFlight];
         held_by(page, held);
#pragma unroll
         for (int k = 0; k < kReleaseFlight; ++k) {
           const bool mine = held[k] == s - kReleaseMark;
           n += __popc(__ballot_sync(0xffffffffu, mine));
           if (out != nullptr && mine) *out |= 1u << k;
         }
       },
       [&](int u) {
         if (lane < ctas) st_cluster(counts_addr + 4u * static_cast<uint32_t>(u), lane, n);
       });
  cluster_barrier();

  int64_t all = 0;
  for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
    const int u = u0 + tid;
    const int64_t to = block_scan(u < units ? counts[u] : 0, all, sums);
    if (u < units) counts[u] = static_cast<int32_t>(to);  // at most num_blocks
  }
  __syncthreads();
  const int64_t top = free_now + all;  // stack height if nothing is dropped
  if (rank == 0 && tid == 0) {
    *p.free_count_out = static_cast<int32_t>(min(top, static_cast<int64_t>(p.free_capacity)));
    if (p.dropped_count != nullptr && top > p.free_capacity)
      atomicAdd(p.dropped_count, static_cast<int32_t>(top - p.free_capacity));
  }
  int64_t at = 0;  // one above the next page's slot
  walk([&](int u) { at = top - (u > 0 ? counts[u - 1] : 0); },
       [&](int s, const int32_t(&page)[kReleaseFlight], uint32_t* known) {
         int32_t held[kReleaseFlight] = {};
         if (known == nullptr) held_by(page, held);
#pragma unroll
         for (int k = 0; k < kReleaseFlight; ++k) {
           const bool mine = known != nullptr ? (*known >> k) & 1u : held[k] == s - kReleaseMark;
           const uint32_t live = __ballot_sync(0xffffffffu, mine);
           const int64_t slot = at - 1 - __popc(live & ((1u << lane) - 1));
           if (mine && slot < p.free_capacity) p.free_pages[slot] = page[k];
           // nobody else takes the 0 for its mark
           if (mine) p.page_shares_out[page[k]] = 0;
           at -= __popc(live);
         }
       },
       nothing);
  cluster_barrier();  // every length has been read
  for (int s = static_cast<int>(rank) * kPlanThreads + tid; s < p.num_seqs;
       s += static_cast<int>(ctas) * kPlanThreads)
    p.seq_lens_out[s] = begin[s] >= 0 ? __ldg(p.keep_lens + s) : p.seq_lens[s];
}

// ---------------------------------------------------------------------- compact
struct CompactParams {
  const int32_t* seq_lens;
  int32_t num_seqs;
  const int32_t* block_table;
  int32_t max_blocks;
  PageSize page;
  const int32_t* page_shares;
  int32_t num_blocks;
  const int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int32_t max_moves;
  int32_t* block_table_out;
  int32_t* page_shares_out;
  int32_t* free_pages_out;
  int32_t* free_count_out;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* pages_end;
  // workspace
  uint32_t* used;   // a bit a page: in a table
  uint32_t* idle;   // a bit a page: on the stack
  int32_t* moved;   // [num_blocks] the page's new id
  int2* ranks;      // used and free pages before a word of the bit maps
  int32_t words;    // of a bit map
};

// Every pass over the tables and the pools' metadata is a launch over the whole
// device; the ranks between them are one CTA's.
__global__ void __launch_bounds__(kPlanThreads) compact_clear_kernel(const CompactParams p) {
  cudaTriggerProgrammaticLaunchCompletion();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  for (int64_t w = first; w < p.words; w += stride) p.used[w] = p.idle[w] = 0u;
  if (first == 0 && p.pages_end != nullptr) *p.pages_end = 0;
  for (int64_t i = first; i < p.num_blocks; i += stride) p.moved[i] = static_cast<int32_t>(i);
  if (p.page_shares_out != p.page_shares)
    copy_ints(p.page_shares, p.page_shares_out, p.num_blocks, first, stride);
}

__global__ void __launch_bounds__(kRowThreads) compact_mark_kernel(const CompactParams p, int32_t chunks) {
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int32_t count = min(max(__ldg(p.free_count), 0), p.free_capacity);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; i < count;
       i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
    const int32_t page = __ldg(p.free_pages + i);
    if (page >= 0 && page < p.num_blocks) atomicOr(p.idle + (page >> 5), 1u << (page & 31));
  }
  const int64_t units = static_cast<int64_t>(p.num_seqs) * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int32_t s = static_cast<int32_t>(u / chunks);
    const int32_t b0 = static_cast<int32_t>(u - static_cast<int64_t>(s) * chunks) * kRowChunk;
    const int32_t end = min(p.page.blocks(__ldg(p.seq_lens + s)), p.max_blocks);
    const int32_t* row = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
    int32_t page[kRowChunk / kRowThreads];
#pragma unroll
    for (int k = 0; k < kRowChunk / kRowThreads; ++k) {
      const int32_t b = b0 + k * kRowThreads + threadIdx.x;
      page[k] = b < end ? __ldg(row + b) : -1;
    }
#pragma unroll
    for (int k = 0; k < kRowChunk / kRowThreads; ++k)
      if (page[k] >= 0 && page[k] < p.num_blocks)
        atomicOr(p.used + (page[k] >> 5), 1u << (page[k] & 31));
  }
}

// The moves: used page number i from the top to free page number i from the
// bottom, as long as that is downwards. One cluster. Every CTA sums up all words
// of the bit maps (a thread has consecutive ones) and keeps the sums before each
// 32 words of its share; then a warp takes a word at a time, a lane a page.
__global__ void __launch_bounds__(kPlanThreads) compact_rank_kernel(const CompactParams p) {
  __shared__ int64_t sums[32];
  __shared__ int32_t sh_moves, sh_end;
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cta_rank(), ctas = cluster_size();
  // the CTA's share of the words, in whole warps' turns
  const int32_t share = (p.words + static_cast<int32_t>(ctas) - 1) / static_cast<int32_t>(ctas);
  const int32_t own0 = min(static_cast<int64_t>(rank) * share, static_cast<int64_t>(p.words));
  const int32_t own1 = min(own0 + static_cast<int64_t>(share), static_cast<int64_t>(p.words));
  auto words_at = [&](int32_t w, uint32_t& used, uint32_t& idle) {
    used = __ldcg(p.used + w);
    idle = __ldcg(p.idle + w) & ~used;  // a page of a table is not free
  };
  // used and free pages before the share, and in all words
  // (a pair of sums below 2^31 in one word: a block's sum takes half a microsecond)
  auto both = [](int used, int idle) { return (static_cast<int64_t>(used) << 32) + idle; };
  int64_t before = 0, all = 0;
  {
    int64_t b = 0, a = 0;
    for (int32_t w = tid; w < p.words; w += kPlanThreads) {
      uint32_t used, idle;
      words_at(w, used, idle);
      const int64_t n = both(__popc(used), __popc(idle));
      a += n;
      if (w < own0) b += n;
    }
    if (ctas > 1) block_scan(b, before, sums);
    block_scan(a, all, sums);
  }
  const int32_t U = static_cast<int32_t>(all >> 32), F = static_cast<int32_t>(all);
  const int32_t most = min(min(U, F), p.max_moves);
  if (tid == 0) sh_moves = sh_end = 0;
  // ranks of the first pages of each word of the share
  for (int32_t w0 = own0; w0 < own1; w0 += kPlanThreads) {
    const int32_t w = w0 + tid;
    uint32_t used = 0, idle = 0;
    if (w < own1) words_at(w, used, idle);
    const int64_t n = both(__popc(used), __popc(idle)), to = block_scan(n, before, sums) - n;
    if (w < own1) p.ranks[w] = make_int2(static_cast<int32_t>(to >> 32), static_cast<int32_t>(to));
  }
  __syncthreads();
  // f(page, whether it is used or free, its rank among those from the top or the bottom, the others' rank)
  auto each = [&](auto&& f) {
    for (int32_t w = own0 + warp; w < own1; w += kPlanWarps) {
      uint32_t used, idle;
      words_at(w, used, idle);
      const int2 r = p.ranks[w];
      const uint32_t below = (1u << lane) - 1u;
      const int32_t nu = r.x + __popc(used & below), ni = r.y + __popc(idle & below);
      // used pages from this one up, free pages below this one
      f(32 * w + lane, (used >> lane) & 1u, (idle >> lane) & 1u, U - nu, ni);
    }
  };
  each([&](int32_t page, bool used, bool idle, int32_t up, int32_t below) {
    if (idle && below < most) p.copy_dst[below] = page;
    if (used && up - 1 < most) p.copy_src[up - 1] = page;
  });
  cluster_barrier();
  int down = 0;
  for (int32_t i = tid; i < most; i += kPlanThreads) down += __ldcg(p.copy_dst + i) < __ldcg(p.copy_src + i);
  if (down > 0) atomicAdd(&sh_moves, down);
  __syncthreads();
  const int32_t m = sh_moves;
  cluster_barrier();  // every CTA has counted: the list may end now
  int32_t end = 0;
  each([&](int32_t page, bool used, bool idle, int32_t up, int32_t below) {
    // the stack: all free pages, the lowest on top
    if (used) {
      if (up - 1 < m) p.free_pages_out[up - 1 + min(F - m, F - below)] = page;
      else end = page + 1;
    } else if (idle) {
      if (below >= m) p.free_pages_out[F - 1 - below + min(m, up)] = page;
      else end = page + 1;
    }
  });
  if (end > 0) atomicMax(&sh_end, end);
  // 64 bits: the lists may be as long as an int32 counts
  for (int64_t i = static_cast<int64_t>(rank) * kPlanThreads + tid; i < p.max_moves;
       i += static_cast<int64_t>(ctas) * kPlanThreads) {
    if (i < m) {
      const int32_t from = __ldcg(p.copy_src + i), to = __ldcg(p.copy_dst + i);
      p.moved[from] = to;
      p.page_shares_out[to] = p.page_shares_out[from];
      p.page_shares_out[from] = 0;
    } else {
      p.copy_src[i] = p.copy_dst[i] = -1;
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (rank == 0) *p.free_count_out = F;
    if (p.pages_end != nullptr && sh_end > 0) atomicMax(p.pages_end, sh_end);
  }
}

__global__ void __launch_bounds__(kRowThreads) compact_table_kernel(const CompactParams p, int32_t chunks) {
  cudaGridDependencySynchronize();
  const bool same = p.block_table_out == p.block_table;
  const int64_t units = static_cast<int64_t>(p.num_seqs) * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int32_t s = static_cast<int32_t>(u / chunks);
    const int32_t b0 = static_cast<int32_t>(u - static_cast<int64_t>(s) * chunks) * kRowChunk;
    const int32_t end = min(p.page.blocks(__ldg(p.seq_lens + s)), p.max_blocks);
    const int64_t row = static_cast<int64_t>(s) * p.max_blocks;
    int32_t page[kRowChunk / kRowThreads], to[kRowChunk / kRowThreads];
#pragma unroll
    for (int k = 0; k < kRowChunk / kRowThreads; ++k) {
      const int32_t b = b0 + k * kRowThreads + threadIdx.x;
      page[k] = b < p.max_blocks ? p.block_table[row + b] : -1;
    }
#pragma unroll
    for (int k = 0; k < kRowChunk / kRowThreads; ++k) {
      const int32_t b = b0 + k * kRowThreads + threadIdx.x;
      const bool live = b < end && page[k] >= 0 && page[k] < p.num_blocks;
      to[k] = live ? __ldcg(p.moved + page[k]) : page[k];
    }
#pragma unroll
    for (int k = 0; k < kRowChunk / kRowThreads; ++k) {
      const int32_t b = b0 + k * kRowThreads + threadIdx.x;
      if (b < p.max_blocks && (!same || to[k] != page[k])) p.block_table_out[row + b] = to[k];
    }
  }
}

// ------------------------------------------------------------------------- copy
// Pages are cut into equal segments of at most 16 KB, a CTA's at a time: each
// thread has four 16-byte loads under way, eight CTAs an SM. A CTA reads the
// page ids of all its units ahead (256 at a time) and keeps those that have a
// page to copy, so that the others cost no memory latency each.
__global__ void __launch_bounds__(kRowThreads)
    copy_pages_kernel(const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                      int32_t num_copies, uint8_t* cache, int64_t num_blocks, int64_t stride,
                      int64_t page_bytes, int32_t segments, int64_t segment_bytes,
                      int32_t* invalid_count) {
  __shared__ int32_t from[kRowThreads], to[kRowThreads], part[kRowThreads];
  __shared__ int32_t live;
  const int64_t units = static_cast<int64_t>(num_copies) * segments;
  for (int64_t u0 = blockIdx.x; u0 < units; u0 += static_cast<int64_t>(gridDim.x) * kRowThreads) {
    const int64_t mine = u0 + static_cast<int64_t>(threadIdx.x) * gridDim.x;
    if (threadIdx.x == 0) live = 0;
    __syncthreads();  // also: the units before have been read
    if (mine < units) {
      const int64_t i = mine / segments;
      const int32_t seg = static_cast<int32_t>(mine - i * segments);
      const int32_t a = __ldg(src + i), b = __ldg(dst + i);
      if (a != -1 && b != -1) {
        if (a < 0 || b < 0 || a >= num_blocks || b >= num_blocks) {
          if (invalid_count != nullptr && seg == 0) atomicAdd(invalid_count, 1);
        } else if (a != b) {
          const int at = atomicAdd(&live, 1);  // in any order: the copies are independent
          from[at] = a;
          to[at] = b;
          part[at] = seg;
        }
      }
    }
    __syncthreads();
    const int n = live;
    for (int k = 0; k < n; ++k) {
      const int64_t lo = part[k] * segment_bytes;
      const int64_t hi = min(lo + segment_bytes, page_bytes);
      const uint8_t* s = cache + from[k] * stride;
      uint8_t* d = cache + to[k] * stride;
      for (int64_t at = lo + 16 * threadIdx.x; at < hi; at += 16 * kRowThreads * kCopyVecs) {
        uint4 v[kCopyVecs];
#pragma unroll
        for (int x = 0; x < kCopyVecs; ++x)
          if (at + 16 * kRowThreads * x < hi)
            v[x] = *reinterpret_cast<const uint4*>(s + at + 16 * kRowThreads * x);
#pragma unroll
        for (int x = 0; x < kCopyVecs; ++x)
          if (at + 16 * kRowThreads * x < hi)
            *reinterpret_cast<uint4*>(d + at + 16 * kRowThreads * x) = v[x];
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------- host
// A launch that may start while the one before it still runs, and waits for it itself.
template <typename... Args>
int32_t launch_after(void (*kernel)(Args...), unsigned grid, unsigned threads, cudaStream_t stream,
                     unsigned cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  return NVFP4_MLA_OK;
}

// CTAs of a release's cluster: 16 where the device runs such a cluster with the most shared
// memory that a call asks for, else 8; asked once a device.
constexpr size_t kReleaseMost = kReleaseBytes * NVFP4_MLA_MAX_PLAN_SEQS + 4 * kReleaseUnits;
int release_cluster(int device) {
  const void* kernel = reinterpret_cast<const void*>(release_kernel);
  constexpr size_t smem = kReleaseMost;
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int n = device < kDevices ? known[device].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    n = kMaxCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) ==
            cudaSuccess &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) == cudaSuccess && fit > 0)
      n = 16;
    cudaGetLastError();
    if (device < kDevices) known[device].store(n, std::memory_order_relaxed);
  }
  return n;
}

unsigned row_grid(int64_t rows, int32_t chunks, int sms) {
  const int64_t units = rows * chunks, most = static_cast<int64_t>(sms) * 8;
  return static_cast<unsigned>(units < 1 ? 1 : units < most ? units : most);
}
int32_t row_chunks(int32_t max_blocks) {  // of up to 2^31 - 1 entries
  return static_cast<int32_t>((int64_t{max_blocks} + kRowChunk - 1) / kRowChunk);
}

size_t bitmap_words(int64_t num_blocks) { return static_cast<size_t>((num_blocks + 127) / 128 * 4); }

}  // namespace
}  // namespace nvfp4_mla

using namespace nvfp4_mla;

extern "C" int32_t nvfp4_mla_fork(const int32_t* src_seqs, const int32_t* dst_seqs,
                                  const int32_t* fork_lens, int32_t num_forks,
                                  const int32_t* seq_lens, int32_t num_seqs, int32_t* block_table,
                                  int32_t max_blocks_per_seq, int32_t page_size,
                                  const int32_t* page_shares, int32_t num_blocks,
                                  const int32_t* free_pages, int32_t free_capacity,
                                  const int32_t* free_count, int32_t* seq_lens_out,
                                  int32_t* page_shares_out, int32_t* free_count_out,
                                  int32_t* shared_blocks, int32_t* copy_src, int32_t* copy_dst,
                                  int32_t* refused_count, void* stream) {
  if (!plan_shape_ok(num_seqs, max_blocks_per_seq, page_size, free_capacity) || num_forks < 0 ||
      num_forks > NVFP4_MLA_MAX_PLAN_SEQS || num_blocks < 1)
    return NVFP4_MLA_ERR_SHAPE;
  if (!seq_lens || !block_table || !page_shares || !free_count || !seq_lens_out ||
      !page_shares_out || !free_count_out || (free_capacity > 0 && !free_pages) ||
      (num_forks > 0 && (!src_seqs || !dst_seqs || !fork_lens || !shared_blocks || !copy_src || !copy_dst)))
    return NVFP4_MLA_ERR_NULL;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;
  const ForkParams p = {src_seqs,    dst_seqs,  fork_lens,  num_forks,      seq_lens,
                        num_seqs,    block_table, max_blocks_per_seq, page_division(page_size),
                        page_shares, num_blocks, free_pages, free_capacity, free_count,
                        seq_lens_out, page_shares_out, free_count_out, shared_blocks, copy_src,
                        copy_dst,    refused_count};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = 4 * static_cast<size_t>(num_seqs);
  // the same limit in every call (it is the process's)
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(reinterpret_cast<const void*>(fork_plan_kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           4 * NVFP4_MLA_MAX_PLAN_SEQS) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  unsigned grid = 1;
  if (page_shares_out != page_shares) {
    const int64_t copying = (static_cast<int64_t>(num_blocks) + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    grid += static_cast<unsigned>(copying < sms ? copying : sms);
  }
  fork_plan_kernel<<<grid, kPlanThreads, smem, s>>>(p);
  if (int32_t st = launch_status()) return st;
  if (num_forks == 0) return NVFP4_MLA_OK;
  const int32_t chunks = row_chunks(max_blocks_per_seq);
  return launch_after(fork_share_kernel, row_grid(num_forks, chunks, sms), kRowThreads, s, 1, p, chunks);
}

extern "C" int32_t nvfp4_mla_release(const int32_t* keep_lens, const int32_t* seq_lens,
                                     int32_t num_seqs, const int32_t* block_table,
                                     int32_t max_blocks_per_seq, int32_t page_size,
                                     const int32_t* page_shares, int32_t num_blocks,
                                     int32_t* free_pages, int32_t free_capacity,
                                     const int32_t* free_count, int32_t* seq_lens_out,
                                     int32_t* page_shares_out, int32_t* free_count_out,
                                     int32_t* dropped_count, int32_t* refused_count, void* stream) {
  if (!plan_shape_ok(num_seqs, max_blocks_per_seq, page_size, free_capacity) || num_blocks < 1)
    return NVFP4_MLA_ERR_SHAPE;
  if (!keep_lens || !seq_lens || !block_table || !page_shares || !free_count || !seq_lens_out ||
      !page_shares_out || !free_count_out || (free_capacity > 0 && !free_pages))
    return NVFP4_MLA_ERR_NULL;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;
  const ReleaseParams p = {keep_lens,   seq_lens,   num_seqs,   block_table,   max_blocks_per_seq,
                           page_division(page_size), page_shares, num_blocks, free_pages,
                           free_capacity, free_count, seq_lens_out, page_shares_out, free_count_out,
                           dropped_count, refused_count};
  const size_t smem = kReleaseBytes * static_cast<size_t>(num_seqs) + 4 * kReleaseUnits;
  // a table that 32 warps walk in one round needs no cluster
  const bool small = static_cast<int64_t>(num_seqs) * row_chunks(max_blocks_per_seq) <= kPlanWarps / 4 &&
                     page_shares_out == page_shares;
  // Its scattered accesses to the counts are what the SMs of a cluster take their
  // time for: sixteen CTAs, where the device holds such a cluster.
  const int ctas = small ? 1 : release_cluster(dev);
  return launch_cluster_smem(release_kernel, p, ctas, smem, kReleaseMost, static_cast<cudaStream_t>(stream));
}

extern "C" size_t nvfp4_mla_compact_workspace_size(int32_t num_blocks) {
  if (num_blocks < 1) return SIZE_MAX;
  return (2 * 4 + sizeof(int2)) * bitmap_words(num_blocks) + 4 * static_cast<size_t>(num_blocks);
}

extern "C" int32_t nvfp4_mla_compact(const int32_t* seq_lens, int32_t num_seqs,
                                     const int32_t* block_table, int32_t max_blocks_per_seq,
                                     int32_t page_size, const int32_t* page_shares,
                                     int32_t num_blocks, const int32_t* free_pages,
                                     int32_t free_capacity, const int32_t* free_count,
                                     int32_t max_moves, int32_t* block_table_out,
                                     int32_t* page_shares_out, int32_t* free_pages_out,
                                     int32_t* free_count_out, int32_t* copy_src, int32_t* copy_dst,
                                     int32_t* pages_end, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (!plan_shape_ok(num_seqs, max_blocks_per_seq, page_size, free_capacity) || num_blocks < 1 ||
      max_moves < 0)
    return NVFP4_MLA_ERR_SHAPE;
  if (!seq_lens || !block_table || !page_shares || !free_count || !block_table_out ||
      !page_shares_out || !free_count_out || (free_capacity > 0 && (!free_pages || !free_pages_out)) ||
      (max_moves > 0 && (!copy_src || !copy_dst)))
    return NVFP4_MLA_ERR_NULL;
  if (!workspace || workspace_bytes < nvfp4_mla_compact_workspace_size(num_blocks))
    return NVFP4_MLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return NVFP4_MLA_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;
  const size_t words = bitmap_words(num_blocks);
  uint32_t* used = static_cast<uint32_t*>(workspace);
  const CompactParams p = {seq_lens,       num_seqs,        block_table,    max_blocks_per_seq,
                           page_division(page_size), page_shares, num_blocks, free_pages,
                           free_capacity,  free_count,      max_moves,      block_table_out,
                           page_shares_out, free_pages_out, free_count_out, copy_src,
                           copy_dst,       pages_end,       used,           used + words,
                           reinterpret_cast<int32_t*>(used + 4 * words),
                           reinterpret_cast<int2*>(used + 2 * words), static_cast<int32_t>(words)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t clearing = (static_cast<int64_t>(num_blocks) + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  compact_clear_kernel<<<static_cast<unsigned>(clearing < sms ? clearing : sms), kPlanThreads, 0, s>>>(p);
  if (int32_t st = launch_status()) return st;
  const int32_t chunks = row_chunks(max_blocks_per_seq);
  const unsigned grid = row_grid(num_seqs, chunks, sms);
  if (int32_t st = launch_after(compact_mark_kernel, grid, kRowThreads, s, 1, p, chunks)) return st;
  // a CTA for each 32 warps' words, as far as a cluster goes
  const unsigned ranks = words <= kPlanWarps ? 1 : kMaxCluster;
  if (int32_t st = launch_after(compact_rank_kernel, ranks, kPlanThreads, s, ranks, p)) return st;
  return launch_after(compact_table_kernel, grid, kRowThreads, s, 1, p, chunks);
}

extern "C" int32_t nvfp4_mla_copy_pages(const int32_t* copy_src, const int32_t* copy_dst,
                                        int32_t num_copies, void* cache, int64_t num_blocks,
                                        int64_t block_stride_bytes, int64_t page_bytes,
                                        int32_t* invalid_count, void* stream) {
  if (num_copies < 0) return NVFP4_MLA_ERR_SHAPE;
  if (num_copies == 0) return NVFP4_MLA_OK;
  if (!copy_src || !copy_dst || !cache) return NVFP4_MLA_ERR_NULL;
  if (num_blocks < 1 || num_blocks > INT32_MAX || page_bytes < 1 || block_stride_bytes < page_bytes ||
      block_stride_bytes > INT64_MAX / num_blocks)
    return NVFP4_MLA_ERR_SHAPE;
  if (!aligned16(cache) || (block_stride_bytes & 15) || (page_bytes & 15)) return NVFP4_MLA_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;
  constexpr int64_t kRound = 16 * kRowThreads * kCopyVecs;  // what a CTA has under way
  const int64_t segments = (page_bytes + kRound - 1) / kRound;
  if (segments > INT32_MAX) return NVFP4_MLA_ERR_SHAPE;
  const int64_t segment_bytes = ((page_bytes + segments - 1) / segments + 15) / 16 * 16;
  copy_pages_kernel<<<row_grid(num_copies, static_cast<int32_t>(segments), sms), kRowThreads, 0,
                      static_cast<cudaStream_t>(stream)>>>(
      copy_src, copy_dst, num_copies, static_cast<uint8_t*>(cache), num_blocks, block_stride_bytes,
      page_bytes, static_cast<int32_t>(segments), segment_bytes, invalid_count);
  return launch_status();
}
