// plan.cu -- block tables and slot maps of a serving step, from request lengths.
//
// nvfp4_mla_plan_step: two prefix sums over the sequences (pages needed,
// tokens wanted) decide who is served, then every token row is filled in.
// nvfp4_mla_truncate: a count of returned pages per sequence, one prefix sum,
// then the pages are pushed. Both work on a few kilobytes to a few megabytes
// in one launch of a thread-block cluster and are bound by latency: their
// dependent global loads (lengths, then page ids) and the cluster's barriers.
// The plan's prefix sums are computed by every CTA of the cluster over all
// sequences, which costs less than exchanging partial sums; its in-place
// updates wait for the cluster barrier behind which nobody reads the old
// lengths any more. With many token rows their index arithmetic bounds it
// (eight SMs work on them).
//
// Measured (GB300, device time): 66 rows of 66 sequences 5.4 us, 131072 rows of
// 1021 sequences 16.5 us (2.1 MB, 0.3 us at the copy rate); drafts of 66
// sequences taken back 4.6 us, a quarter of 1021 sequences released 11.5 us.
#include "plan_common.cuh"

namespace nvfp4_mla {
namespace {

// Dynamic shared memory a sequence, beside the 256 bytes of a scan's sums.
constexpr size_t kPlanBytes = 12, kTruncateBytes = 4;
static_assert(kPlanBytes * NVFP4_MLA_MAX_PLAN_SEQS + 256 <= kMaxSharedBytes, "shared memory");

struct PlanParams {
  const int32_t* new_lens;
  const int32_t* seq_lens;
  int32_t num_seqs;
  int32_t* block_table;
  int32_t max_blocks;
  PageSize page;
  const int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int32_t max_tokens;
  int32_t* seq_lens_out;
  int32_t* free_count_out;
  int32_t* seq_ids;
  int32_t* positions;
  int64_t* slots;
  int32_t* cu_tokens;
  int32_t* refused_count;
};

// Number of entries of end[0..n) that are <= t (32-way search by one warp).
__device__ __forceinline__ int warp_upper_bound(const int32_t* end, int n, int t, int lane) {
  int lo = 0, hi = n;  // the answer is in [lo, hi]
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;  // last entry of lane's part
    const int le = __popc(__ballot_sync(0xffffffffu, i < hi && end[i] <= t));
    lo += le * step;
    hi = min(hi, lo + step);
  }
  const int i = lo + lane;
  return lo + __popc(__ballot_sync(0xffffffffu, i < hi && end[i] <= t));
}

// kAtOnce: 32 token rows each that a warp has under way together.
template <int kAtOnce>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t dyn[];
  int32_t* end = dyn;                  // [num_seqs] tokens up to and with sequence s
  int32_t* first = dyn + p.num_seqs;   // [num_seqs] pages handed out before sequence s
  int32_t* lens = first + p.num_seqs;  // [num_seqs] length before the step
  __shared__ int64_t sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cta_rank(), ctas = cluster_size();
  // an ordinary load: the count may be replaced below
  const int32_t free_now = min(max(*p.free_count, 0), p.free_capacity);
  const int64_t room = static_cast<int64_t>(p.max_blocks) * p.page.size;

  int64_t pages_asked = 0, tokens_asked = 0;  // carries of the two prefix sums
  int64_t pages_taken = 0;
  int refused = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t len = 0, n = 0;
    if (s < p.num_seqs) {
      len = p.seq_lens[s];
      n = p.new_lens[s];
    }
    const bool fits = n >= 0 && len >= 0 && len + n <= room;
    const int64_t need = fits ? p.page.blocks(static_cast<int32_t>(len + n)) -
                                    p.page.blocks(static_cast<int32_t>(len))
                              : 0;
    const int64_t pages_to = block_scan(need, pages_asked, sums);
    const bool paged = fits && (need == 0 || pages_to <= free_now);
    const int64_t tokens_to = block_scan(paged ? n : 0, tokens_asked, sums);
    const bool served = paged && (n == 0 || tokens_to <= p.max_tokens);
    // Who is served with pages (with tokens) is a prefix of those that ask for
    // any, so the sums over the askers are the sums over the served before s.
    if (s < p.num_seqs) {
      lens[s] = static_cast<int32_t>(len);
      first[s] = static_cast<int32_t>(served && need > 0 ? pages_to - need : 0);
      end[s] = static_cast<int32_t>(served && n > 0 ? tokens_to : -1);
      if (!served && n != 0) ++refused;
    }
    const int64_t took = served ? need : 0;
    // running total of pages handed out
    int64_t r = took;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) r += __shfl_xor_sync(0xffffffffu, r, d);
    pages_taken += r;  // per warp; summed below
  }
  __syncthreads();
  if (lane == 0) sums[warp] = pages_taken;
  __syncthreads();
  int64_t all_taken = sums[lane];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) all_taken += __shfl_xor_sync(0xffffffffu, all_taken, d);
  __syncthreads();
  // end[s] of a sequence without tokens: that of the last served one before it
  int32_t carry = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int32_t v = s < p.num_seqs ? end[s] : -1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = max(v, o);
    }
    __syncthreads();
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int32_t w = static_cast<int32_t>(sums[lane]);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w = max(w, o);
    }
    const int32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    const int32_t total = __shfl_sync(0xffffffffu, w, 31);
    v = max(max(v, carry), warp > 0 ? before : 0);
    carry = max(carry, total);
    if (s < p.num_seqs) end[s] = v;
  }
  __syncthreads();
  // Every CTA has read the lengths and the page count; they may be replaced.
  cluster_barrier();

  for (int s = rank * kPlanThreads + tid; s < p.num_seqs; s += ctas * kPlanThreads) {
    const int32_t begin = s > 0 ? end[s - 1] : 0;
    p.seq_lens_out[s] = lens[s] + (end[s] - begin);
    if (p.cu_tokens != nullptr) p.cu_tokens[s + 1] = end[s];
  }
  if (rank == 0) {
    if (tid == 0) {
      if (p.cu_tokens != nullptr) p.cu_tokens[0] = 0;
      *p.free_count_out = free_now - static_cast<int32_t>(all_taken);
    }
    if (p.refused_count != nullptr && refused > 0) atomicAdd(p.refused_count, refused);
  }

  // Token rows: a warp takes 32 * kAtOnce consecutive ones, so that one search
  // serves most of them and their page ids are on their way together. The first
  // token of a fresh page also enters that page into the table.
  const int32_t total = end[p.num_seqs - 1];
  for (int64_t w0 = (static_cast<int64_t>(rank) * kPlanWarps + warp) * (32 * kAtOnce);
       w0 < p.max_tokens; w0 += static_cast<int64_t>(ctas) * kPlanThreads * kAtOnce) {
    int32_t seq[kAtOnce], pos[kAtOnce], row[kAtOnce], page[kAtOnce];
    int32_t* fresh_entry[kAtOnce];
    int at = w0 < total ? warp_upper_bound(end, p.num_seqs, static_cast<int32_t>(w0), lane) : 0;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t t0 = w0 + u * 32;
      seq[u] = pos[u] = page[u] = -1;
      row[u] = 0;
      fresh_entry[u] = nullptr;
      if (t0 >= total) continue;
      if (end[at] <= t0)
        at = warp_upper_bound(end, p.num_seqs, static_cast<int32_t>(t0), lane);
      const int32_t t = static_cast<int32_t>(t0) + lane;
      if (t >= total) continue;
      int s = at;
      if (end[at] <= t) {  // a later sequence's
        int hi = p.num_seqs;
        while (s < hi) {
          const int mid = (s + hi) >> 1;
          if (end[mid] <= t) s = mid + 1;
          else hi = mid;
        }
      }
      const int32_t begin = s > 0 ? end[s - 1] : 0;
      const int32_t len = lens[s];
      seq[u] = s;
      pos[u] = len + (t - begin);
      const int32_t block = p.page.block(pos[u]);
      row[u] = pos[u] - block * p.page.size;
      const int32_t fresh = block - p.page.blocks(len);
      int32_t* entry = p.block_table + static_cast<int64_t>(s) * p.max_blocks + block;
      if (fresh >= 0 && row[u] == 0) fresh_entry[u] = entry;
      // neither the stack nor the entries of blocks that are in use are written
      page[u] = __ldg(fresh >= 0 ? p.free_pages + (free_now - 1 - first[s] - fresh) : entry);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t t = w0 + u * 32 + lane;
      if (fresh_entry[u] != nullptr) *fresh_entry[u] = page[u];
      if (t < p.max_tokens) {
        p.seq_ids[t] = seq[u];
        p.positions[t] = pos[u];
        if (p.slots != nullptr)
          p.slots[t] = page[u] >= 0 ? static_cast<int64_t>(page[u]) * p.page.size + row[u] : -1;
      }
    }
  }
}

struct TruncateParams {
  const int32_t* keep_lens;
  const int32_t* seq_lens;
  int32_t num_seqs;
  const int32_t* block_table;
  int32_t max_blocks;
  PageSize page;
  int32_t* free_pages;
  int32_t free_capacity;
  const int32_t* free_count;
  int32_t* seq_lens_out;
  int32_t* free_count_out;
  int32_t* dropped_count;
};

// A warp per sequence counts the pages it returns, every CTA of the cluster
// gets all counts and sums them up, then the same warp pushes the pages.
__global__ void __launch_bounds__(kPlanThreads) truncate_kernel(const TruncateParams p) {
  extern __shared__ int32_t counts[];  // [num_seqs]; then pages up to and with sequence s
  __shared__ int64_t sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cta_rank(), ctas = cluster_size();
  // an ordinary load: the count may be replaced below
  const int32_t free_now = min(max(*p.free_count, 0), p.free_capacity);
  const uint32_t counts_addr = smem_u32(counts);
  const int first_seq = static_cast<int>(rank) * kPlanWarps + warp;
  const int stride = static_cast<int>(ctas) * kPlanWarps;
  constexpr int kFlight = 8;  // table loads in flight per lane
  cluster_barrier();          // every CTA of the cluster runs: its counts can be written

  auto range = [&](int s, int32_t& b0, int32_t& b1) {
    const int32_t len = p.seq_lens[s], keep = p.keep_lens[s];
    const bool cut = keep >= 0 && keep < len;
    b0 = cut ? p.page.blocks(keep) : 0;
    b1 = cut ? min(p.page.blocks(len), p.max_blocks) : 0;
    return cut ? keep : len;
  };

  for (int s = first_seq; s < p.num_seqs; s += stride) {
    int32_t b0, b1;
    range(s, b0, b1);
    const int32_t* row = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
    int n = 0;
    for (int64_t b = b0; b < b1; b += 32 * kFlight) {
      int32_t page[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        page[u] = b + 32 * u + lane < b1 ? __ldg(row + b + 32 * u + lane) : -1;
#pragma unroll
      for (int u = 0; u < kFlight; ++u) n += __popc(__ballot_sync(0xffffffffu, page[u] >= 0));
    }
    if (lane < ctas) st_cluster(counts_addr + 4u * static_cast<uint32_t>(s), lane, n);
  }
  cluster_barrier();

  int64_t all = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const int64_t to = block_scan(s < p.num_seqs ? counts[s] : 0, all, sums);
    // Page ids are 32-bit and each page is in one table entry, so the sum
    // fits; for a table that breaks this the slots stay in the stack.
    if (s < p.num_seqs) counts[s] = static_cast<int32_t>(min(to, int64_t{INT32_MAX}));
  }
  __syncthreads();
  const int64_t top = free_now + all;  // stack height if nothing is dropped
  if (rank == 0 && tid == 0) {
    *p.free_count_out = static_cast<int32_t>(min(top, static_cast<int64_t>(p.free_capacity)));
    if (p.dropped_count != nullptr && top > p.free_capacity)
      atomicAdd(p.dropped_count, static_cast<int32_t>(top - p.free_capacity));
  }
  for (int s = first_seq; s < p.num_seqs; s += stride) {
    int32_t b0, b1;
    const int32_t len = range(s, b0, b1);
    const int32_t* row = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
    int64_t at = top - (s > 0 ? counts[s - 1] : 0);  // one above the sequence's first page
    for (int64_t b = b0; b < b1; b += 32 * kFlight) {
      int32_t page[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        page[u] = b + 32 * u + lane < b1 ? __ldg(row + b + 32 * u + lane) : -1;
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const uint32_t live = __ballot_sync(0xffffffffu, page[u] >= 0);
        const int64_t slot = at - 1 - __popc(live & ((1u << lane) - 1));
        if (page[u] >= 0 && slot < p.free_capacity) p.free_pages[slot] = page[u];
        at -= __popc(live);
      }
    }
    __syncwarp();  // every lane has read the length
    if (lane == 0) p.seq_lens_out[s] = len;
  }
}

}  // namespace
}  // namespace nvfp4_mla

using namespace nvfp4_mla;

extern "C" int32_t nvfp4_mla_plan_step(
    const int32_t* new_lens, const int32_t* seq_lens, int32_t num_seqs, int32_t* block_table,
    int32_t max_blocks_per_seq, int32_t page_size, const int32_t* free_pages,
    int32_t free_capacity, const int32_t* free_count, int32_t max_tokens, int32_t* seq_lens_out,
    int32_t* free_count_out, int32_t* seq_ids, int32_t* positions, int64_t* slots,
    int32_t* cu_tokens, int32_t* refused_count, void* stream) {
  if (!plan_shape_ok(num_seqs, max_blocks_per_seq, page_size, free_capacity) || max_tokens < 0)
    return NVFP4_MLA_ERR_SHAPE;
  if (!new_lens || !seq_lens || !block_table || !free_count || !seq_lens_out || !free_count_out ||
      (free_capacity > 0 && !free_pages) || (max_tokens > 0 && (!seq_ids || !positions)))
    return NVFP4_MLA_ERR_NULL;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;
  const PlanParams p = {new_lens,       seq_lens,  num_seqs,  block_table, max_blocks_per_seq,
                        page_division(page_size), free_pages, free_capacity, free_count, max_tokens,
                        seq_lens_out,   free_count_out, seq_ids, positions, slots,
                        cu_tokens,      refused_count};
  // A CTA has 32 warps of 32 rows. Past four rounds of them a cluster pays, and
  // a warp takes 128 rows at a time: 131072 rows of 1021 sequences 16.5 us, 25.3
  // with 32. With few rows that leaves warps idle: 66 rows 5.2 us with 32 a
  // warp, 6.2 with 128.
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return max_tokens > 4 * kPlanThreads ? launch_cluster(plan_kernel<4>, p, kMaxCluster, kPlanBytes, s)
                                       : launch_cluster(plan_kernel<1>, p, 1, kPlanBytes, s);
}

extern "C" int32_t nvfp4_mla_truncate(const int32_t* keep_lens, const int32_t* seq_lens,
                                      int32_t num_seqs, const int32_t* block_table,
                                      int32_t max_blocks_per_seq, int32_t page_size,
                                      int32_t* free_pages, int32_t free_capacity,
                                      const int32_t* free_count, int32_t* seq_lens_out,
                                      int32_t* free_count_out, int32_t* dropped_count,
                                      void* stream) {
  if (!plan_shape_ok(num_seqs, max_blocks_per_seq, page_size, free_capacity))
    return NVFP4_MLA_ERR_SHAPE;
  if (!keep_lens || !seq_lens || !block_table || !free_count || !seq_lens_out ||
      !free_count_out || (free_capacity > 0 && !free_pages))
    return NVFP4_MLA_ERR_NULL;
  int dev = 0, sms = 0;
  if (int32_t st = current_device_checked(&dev, &sms)) return st;
  const TruncateParams p = {keep_lens,  seq_lens,      num_seqs,   block_table,  max_blocks_per_seq,
                            page_division(page_size), free_pages, free_capacity, free_count, seq_lens_out,
                            free_count_out, dropped_count};
  const int ctas = num_seqs > kPlanWarps ? kMaxCluster : 1;  // a warp per sequence, as far as 256
  return launch_cluster(truncate_kernel, p, ctas, kTruncateBytes,
                        static_cast<cudaStream_t>(stream));
}
