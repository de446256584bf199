// Host -> HBM gather of the missing chunks (zero-copy kernel variant).
//
// DualDecoder §5.4, GPU-side sparse KV assembly: only the selected KV blocks
// move from host memory into a GPU staging region, where they are laid out
// for attention; the gather on the GPU side avoids the many small host-side
// copies of a CPU gather (§6.4, Fig. 19).  Here one warp copies one chunk of
// K or V (cs rows x 256 bytes, contiguous in both the host tensor and the
// staging slot) with 16-byte loads issued over the host link, eight in
// flight per lane before the stores.
#include "dd_attn.cuh"
#include "dd_kv4.cuh"

namespace dd {

constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads) k_gather(
    const uint4 *__restrict__ Kh, const uint4 *__restrict__ Vh, const int32_t *__restrict__ miss_list,
    const int32_t *__restrict__ miss_count, uint4 *__restrict__ Kst, uint4 *__restrict__ Vst, int64_t max_misses,
    int64_t n_chunks_total, int vec_per_chunk, int32_t *map_out, int32_t *status) {
  pdl_wait();
  pdl_trigger();
  if (load_status(status) != 0) return;
  const int64_t M = min((int64_t)*miss_count, max_misses);
  const int lane = threadIdx.x & 31;
  const int64_t gw = ((int64_t)blockIdx.x * kGatherThreads + threadIdx.x) >> 5;
  const int64_t nw = ((int64_t)gridDim.x * kGatherThreads) >> 5;
  for (int64_t w = gw; w < 2 * M; w += nw) {
    const int64_t m = w >> 1;
    const int half = (int)(w & 1);
    const int32_t packed = miss_list[m];
    if (packed < 0 || packed >= n_chunks_total) {
      if (lane == 0) set_status(status, DD_ERR_DEVICE_CHECK);
      continue;
    }
    if (map_out && half == 0 && lane == 0) map_out[packed] = (int32_t)m;   // prefetch map: chunk -> slot
    const uint4 *src = (half ? Vh : Kh) + (int64_t)packed * vec_per_chunk;
    uint4 *dst = (half ? Vst : Kst) + m * vec_per_chunk;
    for (int i0 = 0; i0 < vec_per_chunk; i0 += 256) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * 32 + lane;
        v[u] = (i < vec_per_chunk) ? ldg_nc(src + i) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * 32 + lane;
        if (i < vec_per_chunk) dst[i] = v[u];
      }
    }
  }
}

static cudaError_t launch_gather_vec(const uint4 *Kh, const uint4 *Vh, const int32_t *miss_list,
                                     const int32_t *miss_count, uint4 *Kst, uint4 *Vst, int64_t max_misses,
                                     int64_t n_chunks_total, int vec_per_chunk, int32_t *status, int sm_count,
                                     cudaStream_t s, int32_t *map_out, int ctas_per_sm) {
  if (max_misses == 0) return cudaSuccess;
  // persistent grid: enough warps to keep the host link busy, never more
  // than the largest possible miss count needs
  const int64_t want_warps = 2 * max_misses;
  int64_t blocks = (want_warps * 32 + kGatherThreads - 1) / kGatherThreads;
  const int64_t cap = (int64_t)sm_count * ctas_per_sm;
  if (blocks > cap) blocks = cap;
  return launch_k(k_gather, dim3((unsigned)blocks), dim3(kGatherThreads), 0, s, Kh, Vh, miss_list, miss_count, Kst,
                  Vst, max_misses, n_chunks_total, vec_per_chunk, map_out, status);
}

cudaError_t launch_gather(const uint4 *Kh, const uint4 *Vh, const int32_t *miss_list, const int32_t *miss_count,
                          uint4 *Kst, uint4 *Vst, int64_t max_misses, int64_t n_chunks_total, int cs,
                          int32_t *status, int sm_count, cudaStream_t s, int32_t *map_out, int ctas_per_sm) {
  return launch_gather_vec(Kh, Vh, miss_list, miss_count, Kst, Vst, max_misses, n_chunks_total, cs * kVecPerRow,
                           status, sm_count, s, map_out, ctas_per_sm);
}

// ------------------------------------------------------------- 4-bit chunks
// Expansion to bf16: one warp per block of 16 rows of K or V; a lane turns the
// four bytes of codes of 8 values (16 lanes a row, two rows an instruction), so
// loads and stores are whole lines.  Bound by the host link (72 bytes a row), or,
// from a home cache in HBM, by the 256 bytes written for each row.
__global__ void __launch_bounds__(kGatherThreads) k_expand4(
    const uint8_t *__restrict__ Kh, const uint8_t *__restrict__ Vh, const int32_t *__restrict__ miss_list,
    const int32_t *__restrict__ miss_count, uint4 *__restrict__ Kst, uint4 *__restrict__ Vst, int64_t max_misses,
    int64_t n_chunks_total, int blocks_per_chunk, int C, int Hkv, const int32_t *__restrict__ k_exp,
    const int32_t *__restrict__ v_exp, int32_t *status) {
  pdl_wait();
  pdl_trigger();
  if (load_status(status) != 0) return;
  const int64_t M = min((int64_t)*miss_count, max_misses);
  const int lane = threadIdx.x & 31;
  const int64_t gw = ((int64_t)blockIdx.x * kGatherThreads + threadIdx.x) >> 5;
  const int64_t nw = ((int64_t)gridDim.x * kGatherThreads) >> 5;
  for (int64_t w = gw; w < 2 * M * blocks_per_chunk; w += nw) {
    const int64_t mb = w >> 1, m = mb / blocks_per_chunk;
    const int half = (int)(w & 1), blk = (int)(mb - m * blocks_per_chunk);
    const int32_t packed = miss_list[m];
    if (packed < 0 || packed >= n_chunks_total) {
      if (lane == 0) set_status(status, DD_ERR_DEVICE_CHECK);
      continue;
    }
    const float mul = pow2i(head_exp(half ? v_exp : k_exp, packed / C % Hkv, status));
    const uint8_t *src = (half ? Vh : Kh) + ((int64_t)packed * blocks_per_chunk + blk) * kBlk4;
    uint4 *dst = (half ? Vst : Kst) + mb * 16 * kVecPerRow + lane;
    uint32_t codes[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) codes[i] = *reinterpret_cast<const uint32_t *>(src + i * 128 + lane * 4);
    // rows 2i and 2i + 1: group (lane & 15) / 2 of row 2i + lane / 16
    uint32_t sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sc[i] = src[kBlk4Scales + (2 * i + (lane >> 4)) * 8 + ((lane & 15) >> 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h[4], o[4];
      e2m1x8_to_half2(codes[i], h);
      const float s = __half2float(__ushort_as_half((uint16_t)(e4m3x2_to_half2(sc[i]) & 0xFFFFu))) * mul;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
        o[e] = cvt_bf16x2(v.x * s, v.y * s);
      }
      dst[i * 32] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

cudaError_t launch_gather4(const uint8_t *Kh, const uint8_t *Vh, const int32_t *miss_list, const int32_t *miss_count,
                           void *Kst, void *Vst, bool expand, const int32_t *k_exp, const int32_t *v_exp,
                           int64_t max_misses, int units, int Hkv, int C, int cs, int32_t *status, int sm_count,
                           cudaStream_t s) {
  if (max_misses == 0) return cudaSuccess;
  const int64_t total = (int64_t)units * C;
  if (!expand)
    return launch_gather_vec(reinterpret_cast<const uint4 *>(Kh), reinterpret_cast<const uint4 *>(Vh), miss_list,
                             miss_count, static_cast<uint4 *>(Kst), static_cast<uint4 *>(Vst), max_misses, total,
                             cs * kRow4 / 16, status, sm_count, s, nullptr, 8);
  const int bpc = cs / 16;
  int64_t blocks = (2 * max_misses * bpc * 32 + kGatherThreads - 1) / kGatherThreads;
  if (blocks > (int64_t)sm_count * 8) blocks = (int64_t)sm_count * 8;
  return launch_k(k_expand4, dim3((unsigned)blocks), dim3(kGatherThreads), 0, s, Kh, Vh, miss_list, miss_count,
                  static_cast<uint4 *>(Kst), static_cast<uint4 *>(Vst), max_misses, total, bpc, C, Hkv, k_exp, v_exp,
                  status);
}

}  // namespace dd
