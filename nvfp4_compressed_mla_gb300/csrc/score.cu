// score.cu -- index scores of every visible position of every query token.
#include "select_common.cuh"

namespace nvfp4_mla {
namespace {

// One thread per position of a tile, the query's dequantised heads in shared
// memory.
__global__ void __launch_bounds__(kScoreTile) score_kernel(const SelectParams p) {
  extern __shared__ float qv[];  // [num_heads][128]
  __shared__ float wmax[4];
  const int32_t t = blockIdx.y;
  const int32_t seen = scored_positions(p, t);
  const int32_t pos0 = blockIdx.x * kScoreTile;
  if (pos0 >= seen) return;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int g = tid; g < p.num_heads * kIndexScales; g += kScoreTile) {
    const uint8_t* src = p.q_index +
                         (static_cast<int64_t>(t) * p.num_heads * kIndexScales + g) * (2 * kGroup);
    const uint4 a = ld_nc_v4(src), b = ld_nc_v4(src + 16);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t lo, hi, h[8];
    float s;
    quantize_group(w, lo, hi, s);
    uint32_t x[4], y[4];
    e2m1x8_to_f16x8(lo, x);
    e2m1x8_to_f16x8(hi, y);
    for (int i = 0; i < 4; ++i) h[i] = x[i], h[4 + i] = y[i];
    for (int i = 0; i < 8; ++i) {
      qv[g * kGroup + 2 * i] = f16_bits_to_f32(static_cast<uint16_t>(h[i])) * s;
      qv[g * kGroup + 2 * i + 1] = f16_bits_to_f32(static_cast<uint16_t>(h[i] >> 16)) * s;
    }
  }
  __syncthreads();
  const int32_t pos = pos0 + tid;
  float score = -INFINITY, smax = 0.f;
  if (pos < seen) {
    const IndexRow at = resolve_index_row(__ldg(p.q_seq + t), pos, p.block_table, p.num_seqs,
                                          p.max_blocks, p.page_size, p.num_blocks,
                                          p.block_stride);
    if (at.page >= 0) {
      const uint8_t* page = p.cache + at.page;
      const uint8_t* sc = page + static_cast<int64_t>(p.page_size) * kIndexCodes +
                          static_cast<int64_t>(at.row) * kIndexScales;
      float k[kIndexDim];
      for (int g = 0; g < kIndexScales; ++g) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(
            page + static_cast<int64_t>(at.row) * kIndexCodes + g * 8));
        const uint8_t byte = __ldg(sc + g) & 0x7Fu;
        const float s = f16_bits_to_f32(static_cast<uint16_t>(e4m3x2_to_f16x2(byte)));
        smax = fmaxf(smax, byte == 0x7Fu ? 448.f : s);
        uint32_t x[4], y[4];
        e2m1x8_to_f16x8(c.x, x);
        e2m1x8_to_f16x8(c.y, y);
        for (int i = 0; i < 4; ++i) {
          k[g * kGroup + 2 * i] = f16_bits_to_f32(static_cast<uint16_t>(x[i])) * s;
          k[g * kGroup + 2 * i + 1] = f16_bits_to_f32(static_cast<uint16_t>(x[i] >> 16)) * s;
          k[g * kGroup + 8 + 2 * i] = f16_bits_to_f32(static_cast<uint16_t>(y[i])) * s;
          k[g * kGroup + 8 + 2 * i + 1] = f16_bits_to_f32(static_cast<uint16_t>(y[i] >> 16)) * s;
        }
      }
      float sum = 0.f;
      for (int j = 0; j < p.num_heads; ++j) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < kIndexDim; ++i) d = fmaf(qv[j * kIndexDim + i], k[i], d);
        d = d < 0.f ? 0.f : d;
        sum = fmaf(__ldg(p.weights + static_cast<int64_t>(t) * p.num_heads + j), d, sum);
      }
      if (!(sum != sum)) score = sum + 0.f;
    }
  }
  const int granule = min(p.block, kMaxGranule);
  for (int d = 1; d < granule; d <<= 1)
    score = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, d));
  if (pos < seen && pos % granule == 0)
    p.scores[t * p.score_stride + pos / granule] = score;
  for (int d = 16; d > 0; d >>= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, d));
  if (lane == 0) wmax[tid >> 5] = smax;
  __syncthreads();
  if (tid == 0)
    p.smax[t * p.tiles + blockIdx.x] = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
}

}  // namespace

int32_t launch_scores(SelectParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  p.score_ctas = 0;
  const size_t smem = static_cast<size_t>(p.num_heads) * kIndexDim * 4;
  if (cudaFuncSetAttribute(score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  score_kernel<<<dim3(static_cast<unsigned>(p.tiles), p.num_q), kScoreTile, smem, stream>>>(p);
  return launch_status();
}

}  // namespace nvfp4_mla
