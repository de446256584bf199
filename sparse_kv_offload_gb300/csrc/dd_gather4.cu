// Gather of missing chunks from a 4-bit home cache (pinned host, or HBM), as they are or
// expanded to bf16 values.
//
// A chunk takes 72 bytes a row instead of 256, and the host link bounds a step whose chunks are
// missing.  20,000 chunks of 16 rows from pinned memory, in any order: bf16 800 us (205 GB/s, a
// copy 210), 4 bits 238 us (194 GB/s), expanded 240 us: 3.4 times as many rows a second.
// 2,000 chunks, where latency begins to count: 98, 40 and 42 us.
#include "dd_attn.cuh"
#include "dd_kv4.cuh"

namespace dd {

constexpr int kThreads4 = 256;

// One warp per chunk of K or V (contiguous on both sides), 16-byte loads, all of a chunk of
// up to 32 rows in flight before the stores.
__global__ void __launch_bounds__(kThreads4) k_gather4(
    const uint4 *__restrict__ Kh, const uint4 *__restrict__ Vh, const int32_t *__restrict__ miss_list,
    const int32_t *__restrict__ miss_count, uint4 *__restrict__ Kst, uint4 *__restrict__ Vst, int64_t max_misses,
    int64_t n_chunks_total, int vec_per_chunk, int32_t *status) {
  pdl_wait();
  pdl_trigger();
  if (load_status(status) != 0) return;
  const int64_t M = min((int64_t)*miss_count, max_misses);
  const int lane = threadIdx.x & 31;
  const int64_t gw = ((int64_t)blockIdx.x * kThreads4 + threadIdx.x) >> 5;
  const int64_t nw = ((int64_t)gridDim.x * kThreads4) >> 5;
  for (int64_t w = gw; w < 2 * M; w += nw) {
    const int64_t m = w >> 1;
    const int half = (int)(w & 1);
    const int32_t packed = miss_list[m];
    if (packed < 0 || packed >= n_chunks_total) {
      if (lane == 0) set_status(status, DD_ERR_DEVICE_CHECK);
      continue;
    }
    const uint4 *src = (half ? Vh : Kh) + (int64_t)packed * vec_per_chunk;
    uint4 *dst = (half ? Vst : Kst) + m * vec_per_chunk;
    for (int i0 = 0; i0 < vec_per_chunk; i0 += 160) {
      uint4 v[5];
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        const int i = i0 + u * 32 + lane;
        v[u] = i < vec_per_chunk ? ldg_nc(src + i) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        const int i = i0 + u * 32 + lane;
        if (i < vec_per_chunk) dst[i] = v[u];
      }
    }
  }
}

// Expansion to bf16: one warp per block of 16 rows of K or V; a lane turns the
// four bytes of codes of 8 values (16 lanes a row, two rows an instruction), so
// loads and stores are whole lines.  Bound by the host link (72 bytes a row), or,
// from a home cache in HBM, by the 256 bytes written for each row: 231 MB in 37 us, 92% of the
// copy rate (every lane loading its own scales 44 us).
__global__ void __launch_bounds__(kThreads4) k_expand4(
    const uint8_t *__restrict__ Kh, const uint8_t *__restrict__ Vh, const int32_t *__restrict__ miss_list,
    const int32_t *__restrict__ miss_count, uint4 *__restrict__ Kst, uint4 *__restrict__ Vst, int64_t max_misses,
    int64_t n_chunks_total, int blocks_per_chunk, int C, int Hkv, const int32_t *__restrict__ k_exp,
    const int32_t *__restrict__ v_exp, int32_t *status) {
  pdl_wait();
  pdl_trigger();
  if (load_status(status) != 0) return;
  const int64_t M = min((int64_t)*miss_count, max_misses);
  const int lane = threadIdx.x & 31;
  const int64_t gw = ((int64_t)blockIdx.x * kThreads4 + threadIdx.x) >> 5;
  const int64_t nw = ((int64_t)gridDim.x * kThreads4) >> 5;
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
    // the block's 128 scales, four a lane, handed round
    const uint32_t four = *reinterpret_cast<const uint32_t *>(src + kBlk4Scales + lane * 4);
    uint32_t sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sc[i] = __shfl_sync(0xffffffffu, four, 4 * i + (lane >> 4) * 2 + ((lane >> 3) & 1)) >> (((lane >> 1) & 3) * 8) & 0xFFu;
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
  const int bpc = cs / 16;
  // no larger than the most misses need; the copy's blocks are all resident at once, of the
  // expansion's five an SM are, and short blocks even out the end (231 MB: 5 an SM 41 us, 8 38,
  // 16 37, 64 39)
  const int64_t most = (int64_t)sm_count * (expand ? 16 : 8);
  int64_t blocks = (2 * max_misses * (expand ? bpc : 1) * 32 + kThreads4 - 1) / kThreads4;
  if (blocks > most) blocks = most;
  if (!expand)
    return launch_k(k_gather4, dim3((unsigned)blocks), dim3(kThreads4), 0, s, reinterpret_cast<const uint4 *>(Kh),
                    reinterpret_cast<const uint4 *>(Vh), miss_list, miss_count, static_cast<uint4 *>(Kst),
                    static_cast<uint4 *>(Vst), max_misses, total, cs * kRow4 / 16, status);
  return launch_k(k_expand4, dim3((unsigned)blocks), dim3(kThreads4), 0, s, Kh, Vh, miss_list, miss_count,
                  static_cast<uint4 *>(Kst), static_cast<uint4 *>(Vst), max_misses, total, bpc, C, Hkv, k_exp, v_exp,
                  status);
}

}  // namespace dd
