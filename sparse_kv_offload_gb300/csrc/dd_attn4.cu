// Attention over a cache held in 4 bits: out = softmax(scale q.K^T) V over the rows
// of the union's chunks that each query selected, K and V decoded on the way.
//
// One CTA per (request, KV head, query vector): its warps take the chunks in
// turn, a lane holds four of a row's 128 values, and each warp keeps a running
// maximum, sum and output; the warps' states are joined at the end with the step's
// own rows.
#include "dd_kv4.cuh"

namespace dd {

namespace {

constexpr int kWarps = 8;

struct Row4 {
  float v[4];
};

// values 4 lane .. 4 lane + 3 of row t of a page
__device__ __forceinline__ Row4 row4(const uint8_t *page, int t, int lane) {
  const uint8_t *blk = page + (t >> 4) * kBlk4;
  const uint32_t c = *reinterpret_cast<const uint16_t *>(blk + (t & 15) * 64 + lane * 2);
  const uint32_t s = blk[kBlk4Scales + (t & 15) * 8 + (lane >> 2)];
  uint32_t h[4];
  e2m1x8_to_half2(c, h);
  const float sc = __half2float(__ushort_as_half((uint16_t)(e4m3x2_to_half2(s) & 0xFFFFu)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h[0]));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h[1]));
  return {{a.x * sc, a.y * sc, b.x * sc, b.y * sc}};
}

__device__ __forceinline__ Row4 row16(const uint16_t *p, int lane) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p + 4 * lane);
  return {{bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)}};
}

__device__ __forceinline__ float dot(const Row4 &a, const Row4 &b) {
  float x = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) x = fmaf(a.v[e], b.v[e], x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

struct State {
  float m = -INFINITY, l = 0.f;
  Row4 o = {{0.f, 0.f, 0.f, 0.f}};
  __device__ __forceinline__ void add(float x, const Row4 &v, float mul) {   // a row of score x and values v * mul
    float mn = fmaxf(m, x);
    if (mn == -INFINITY) {
      if (x == x) return;
      mn = 0.f;   // the first row's score is NaN: so is the result
    }
    const float a = exp2f(m - mn), p = exp2f(x - mn);
    l = l * a + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) o.v[e] = fmaf(o.v[e], a, p * (v.v[e] * mul));
    m = mn;
  }
};

__global__ void __launch_bounds__(kWarps * 32) k_attn4(Attn4Args p) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kD];
  pdl_wait();
  pdl_trigger();
  if (load_status(p.status) != 0) return;
  const int G = p.Hq / p.Hkv, NQ = p.n_q * G;
  const int unit = blockIdx.x / NQ, qv = blockIdx.x - unit * NQ;
  const int b = unit / p.Hkv, g = unit - b * p.Hkv, j = qv / G, h = g * G + qv - j * G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t at = ((int64_t)(b * p.n_q + j) * p.Hq + h) * kD;
  const Row4 q = row16(static_cast<const uint16_t *>(p.q) + at, lane);
  const float sl2 = p.softmax_scale * 1.4426950408889634f;
  const float kmul = pow2i(head_exp(p.k_exp, g, p.status)) * sl2, vmul = pow2i(head_exp(p.v_exp, g, p.status));
  const int64_t page = (int64_t)p.cs * kRow4;
  const int64_t staged = p.miss_count ? min((int64_t)*p.miss_count, p.max_misses) : p.max_misses;
  int n = p.union_cnt[unit];
  if (n < 0 || n > p.umax) {
    set_status(p.status, DD_ERR_DEVICE_CHECK);
    n = n < 0 ? 0 : p.umax;
  }
  State st;
  for (int i = warp; i < n; i += kWarps) {
    const int64_t x = (int64_t)unit * p.umax + i;
    if (p.union_qmask && !((p.union_qmask[x] >> j) & 1)) continue;
    const int64_t slot = p.union_slot[x];
    if (slot >= 0 ? slot >= p.hot_slots : -slot - 1 >= staged) {
      set_status(p.status, DD_ERR_DEVICE_CHECK);
      continue;
    }
    const uint8_t *kp = slot >= 0 ? p.Khot + slot * page : p.Kst + (-slot - 1) * page;
    const uint8_t *vp = slot >= 0 ? p.Vhot + slot * page : p.Vst + (-slot - 1) * page;
    const int64_t left = p.kv_len ? (int64_t)p.kv_len[b] - (int64_t)p.union_idx[x] * p.cs : p.cs;
    const int rows = (int)min((int64_t)p.cs, left);
    for (int t = 0; t < rows; ++t) st.add(dot(q, row4(kp, t, lane)) * kmul, row4(vp, t, lane), vmul);
  }
  if (p.k_tail && warp == 0) {
    for (int t = 0; t <= j; ++t) {
      const int64_t r = ((int64_t)(b * p.n_q + t) * p.Hkv + g) * kD;
      st.add(dot(q, row16(static_cast<const uint16_t *>(p.k_tail) + r, lane)) * sl2,
             row16(static_cast<const uint16_t *>(p.v_tail) + r, lane), 1.f);
    }
  }
  if (lane == 0) s_m[warp] = st.m, s_l[warp] = st.l;
#pragma unroll
  for (int e = 0; e < 4; ++e) s_o[warp][4 * lane + e] = st.o.v[e];
  __syncthreads();
  if (threadIdx.x < kD) {
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w]);
    for (int w = 0; w < kWarps && m != -INFINITY; ++w) {
      const float a = exp2f(s_m[w] - m);
      l += a * s_l[w];
      o += a * s_o[w][threadIdx.x];
    }
    p.out[at + threadIdx.x] = l == 0.f ? 0.f : o / l;
  }
}

}  // namespace

cudaError_t launch_attn4(const Attn4Args &a, cudaStream_t s) {
  const int64_t ctas = (int64_t)a.B * a.Hkv * a.n_q * (a.Hq / a.Hkv);
  return launch_k(k_attn4, dim3((unsigned)ctas), dim3(kWarps * 32), 0, s, a);
}

}  // namespace dd
