// Eviction from the pools by gathered attention weight, and slots for the chunks to come.
//
// A (request, KV head) unit u owns slots u S .. u S + S - 1 of the pool.  With n0 = ceil(kv_len / cs)
// chunks so far and n1 = ceil((kv_len + new_len) / cs) to be, R chunks resident and N of n0 .. n1 - 1
// without a slot, E = clamp(R + N - keep, 0, candidates) chunks leave: those of the smallest weight among the
// resident chunks c with first <= c < n0 - last, the lower chunk first where weights are equal.
// The N new chunks then take free slots, ascending both.
//
// One CTA a unit: weights become order keys in shared memory (a NaN below every number, -0 as
// +0), an 8-bit radix select finds the E-th smallest, and a warp takes a run of chunks, 32 at a
// time, so that ranks are ballots and every access is a whole line.
#include "dd_pages.cuh"

namespace dd {

namespace {

enum : uint8_t { kAbsent = 0, kStays = 1, kMay = 2, kNew = 3 };

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix over the warps of up to three counts of each warp; the totals in t.
struct Counts {
  int a, b, c;
};
__device__ __forceinline__ Counts warp_prefix(Counts v, int (*scratch)[33], Counts &t, int warp, int lane, int warps) {
  if (lane == 0) scratch[0][warp] = v.a, scratch[1][warp] = v.b, scratch[2][warp] = v.c;
  __syncthreads();
  if (warp < 3) {
    const int x = lane < warps ? scratch[warp][lane] : 0, s = warp_incl_scan(x);
    __syncwarp();
    if (lane < warps) scratch[warp][lane] = s - x;
    if (lane == 31) scratch[warp][32] = s;
  }
  __syncthreads();
  const Counts r = {scratch[0][warp], scratch[1][warp], scratch[2][warp]};
  t = {scratch[0][32], scratch[1][32], scratch[2][32]};
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(1024) k_evict(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t *key = sm;                                        // [C]
  uint16_t *free_slot = reinterpret_cast<uint16_t *>(sm);    // [S], then owners [S], once the keys are done with
  const int words = (a.S + 31) / 32;
  const int front = max(a.C, a.S + 1);
  uint32_t *used = sm + front;                               // [words]
  uint8_t *state = reinterpret_cast<uint8_t *>(used + words);   // [C]
  uint16_t *owner = free_slot + a.S;
  __shared__ int scratch[3][33];
  __shared__ uint32_t hist[256];
  __shared__ int s_bad;
  __shared__ uint32_t s_digit, s_rank;

  pdl_wait();
  pdl_trigger();
  if (load_status(a.status) != 0) return;
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int b = u / a.Hkv;
  const int64_t row = (int64_t)u * a.C, base = (int64_t)u * a.S;
  const int kv = a.kv_len[b], more = a.new_len ? a.new_len[b] : 0;
  bool bad = kv < 0 || more < 0 || (int64_t)kv + more > (int64_t)a.C * a.cs;
  const int n0 = bad ? 0 : (kv + a.cs - 1) / a.cs, n1 = bad ? 0 : (kv + more + a.cs - 1) / a.cs;
  const int seg = ((a.C + 31) / 32 + warps - 1) / warps * 32, lo = min(a.C, warp * seg), hi = min(a.C, lo + seg);

  if (tid == 0) s_bad = 0;
  for (int i = tid; i < words; i += blockDim.x) used[i] = 0u;
  __syncthreads();
  Counts n = {0, 0, 0};                                      // resident, new, candidates
  for (int c0 = lo; c0 < hi; c0 += 32) {
    const int c = c0 + lane;
    uint8_t st = kAbsent;
    if (c < hi) {
      const int64_t s = a.resident_slot[row + c];
      if (s >= 0) {
        const int64_t k = s - base;
        // a slot of another unit, or of two chunks
        if (k < 0 || k >= a.S || (atomicOr(&used[k >> 5], 1u << (k & 31)) >> (k & 31) & 1u)) s_bad = 1;
        st = c >= a.first && c < n0 - a.last ? kMay : kStays;
      } else if (c >= n0 && c < n1) {
        st = kNew;
      }
      state[c] = st;
      key[c] = st == kMay ? order_key(a.weight[row + c]) : 0xFFFFFFFFu;
    }
    n.a += __popc(__ballot_sync(0xffffffffu, st == kStays || st == kMay));
    n.b += __popc(__ballot_sync(0xffffffffu, st == kNew));
    n.c += __popc(__ballot_sync(0xffffffffu, st == kMay));
  }
  Counts all;
  warp_prefix(n, scratch, all, warp, lane, warps);
  bad = bad || s_bad != 0;
  if (bad) {
    // left as it was
    if (tid == 0) {
      set_status(a.status, DD_ERR_DEVICE_CHECK);
      if (a.evicted_cnt) a.evicted_cnt[u] = 0;
      if (a.list_cnt) a.list_cnt[u] = 0;
    }
    for (int c = tid; c < a.C; c += blockDim.x) a.resident_out[row + c] = a.resident_slot[row + c];
    return;
  }
  const int leave = min(max(all.a + all.b - a.keep, 0), all.c);

  // the leave-th smallest key of the candidates, and how many equal to it leave
  uint32_t bound = 0u, rank = (uint32_t)leave;               // of those that share the digits found so far
  if (leave > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += blockDim.x) hist[i] = 0u;
      __syncthreads();
      for (int c0 = lo; c0 < hi; c0 += 32) {
        const int c = c0 + lane;
        if (c < hi && state[c] == kMay) {
          const uint32_t k = key[c];
          if (shift == 24 || (k >> (shift + 8)) == (bound >> (shift + 8))) atomicAdd(&hist[k >> shift & 255u], 1u);
        }
      }
      __syncthreads();
      if (warp == 0) {
        uint32_t sum = 0, v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = hist[8 * lane + i], sum += v[i];
        uint32_t before = (uint32_t)warp_incl_scan((int)sum) - sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < rank && rank <= before + v[i]) s_digit = 8 * lane + i, s_rank = rank - before;
          before += v[i];
        }
      }
      __syncthreads();
      bound |= s_digit << shift;
      rank = s_rank;
    }
  }

  // ties at the bound leave in chunk order
  Counts m = {0, 0, 0};
  if (leave > 0)
    for (int c0 = lo; c0 < hi; c0 += 32) {
      const int c = c0 + lane;
      m.a += __popc(__ballot_sync(0xffffffffu, c < hi && state[c] == kMay && key[c] == bound));
    }
  int ties = warp_prefix(m, scratch, all, warp, lane, warps).a;
  m = {0, 0, 0};                                             // leaving, new, staying
  for (int c0 = lo; c0 < hi; c0 += 32) {
    const int c = c0 + lane;
    const uint8_t st = c < hi ? state[c] : (uint8_t)kAbsent;
    bool go = false;
    if (leave > 0) {
      const bool tie = st == kMay && key[c] == bound;
      const uint32_t in = __ballot_sync(0xffffffffu, tie);
      go = st == kMay && (key[c] < bound || (tie && ties + __popc(in & ((1u << lane) - 1u)) < (int)rank));
      ties += __popc(in);
    }
    if (go) {
      const int k = (int)(a.resident_slot[row + c] - base);
      atomicAnd(&used[k >> 5], ~(1u << (k & 31)));
    }
    // (from here on: kMay leaves)
    if (c < hi) state[c] = st == kMay && !go ? (uint8_t)kStays : st;
    m.a += __popc(__ballot_sync(0xffffffffu, go));
    m.b += __popc(__ballot_sync(0xffffffffu, st == kNew));
    m.c += __popc(__ballot_sync(0xffffffffu, st == kStays || (st == kMay && !go)));
  }
  const Counts pre = warp_prefix(m, scratch, all, warp, lane, warps);

  // the free slots, ascending (the keys are done with)
  int taken_by = 0;
  {
    int f = 0;
    uint32_t w = 0;
    for (int i = warp * 32; i < words; i += warps * 32) {    // at most 512 words: one each
      const int k = i + lane;
      if (k < words) {
        w = ~used[k];
        if (k == words - 1 && (a.S & 31)) w &= (1u << (a.S & 31)) - 1u;
      }
      f = __popc(w);
    }
    const int incl = warp_incl_scan(f);
    Counts t, fc = {__shfl_sync(0xffffffffu, incl, 31), 0, 0};
    int at = warp_prefix(fc, scratch, t, warp, lane, warps).a + incl - f;
    taken_by = t.a;
    const int k = warp * 32 + lane;
    while (w) {
      const int bit = __ffs((int)w) - 1;
      w &= w - 1;
      free_slot[at++] = (uint16_t)(32 * k + bit);
    }
    for (int i = tid; i < a.S; i += blockDim.x) owner[i] = 0xFFFFu;
  }
  __syncthreads();
  if (all.b > taken_by && tid == 0) set_status(a.status, DD_ERR_CAPACITY);
  const int given = min(all.b, taken_by);

  // lists need the new chunks that have got a slot: they are behind n0, among the residents there
  int gone = pre.a, fresh = pre.b, stay = pre.c;
  for (int c0 = lo; c0 < hi; c0 += 32) {
    const int c = c0 + lane;
    const uint8_t st = c < hi ? state[c] : (uint8_t)kAbsent;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t in_go = __ballot_sync(0xffffffffu, st == kMay), in_new = __ballot_sync(0xffffffffu, st == kNew),
                   in_stay = __ballot_sync(0xffffffffu, st == kStays);
    const int my_new = fresh + __popc(in_new & below), my_stay = stay + __popc(in_stay & below);
    if (c < hi) {
      const int32_t old = a.resident_slot[row + c];
      int32_t now = -1;
      if (st == kStays) now = old;
      if (st == kNew && my_new < given) now = (int32_t)base + free_slot[my_new];
      a.resident_out[row + c] = now;
      if (now >= 0) {
        owner[now - base] = (uint16_t)c;
        const int at = my_stay + min(my_new, given);
        if (a.list_idx) a.list_idx[(int64_t)u * a.umax + at] = c;
        if (a.list_slot) a.list_slot[(int64_t)u * a.umax + at] = now;
        if (st == kNew && a.last_used) a.last_used[now] = a.step;
      }
      if (st == kMay && a.evicted) a.evicted[base + gone + __popc(in_go & below)] = c;
    }
    gone += __popc(in_go), fresh += __popc(in_new), stay += __popc(in_stay);
  }
  if (tid == 0) {
    if (a.evicted_cnt) a.evicted_cnt[u] = all.a;
    if (a.list_cnt) a.list_cnt[u] = all.c + given;
  }
  __syncthreads();
  if (a.slot_chunk || a.last_used)
    for (int i = tid; i < a.S; i += blockDim.x) {
      const uint16_t c = owner[i];
      if (a.slot_chunk) a.slot_chunk[base + i] = c == 0xFFFFu ? -1 : (int32_t)c;
      if (a.last_used && c == 0xFFFFu) a.last_used[base + i] = -1;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s) {
  const int per = (a.C + 31) / 32;                 // runs of 32 chunks
  const int words = (a.S + 31) / 32, front = a.C > a.S + 1 ? a.C : a.S + 1;
  int threads = 32 * (per < 32 ? (per < 4 ? 4 : per) : 32);
  if (threads < words) threads = (words + 31) / 32 * 32;      // a thread a word of free slots
  const size_t smem = (size_t)(front + words) * 4 + a.C;
  cudaError_t e = set_dyn_smem((const void *)k_evict, smem);
  if (e != cudaSuccess) return e;
  return launch_k(k_evict, dim3(a.units), dim3(threads), smem, s, a);
}

}  // namespace dd
