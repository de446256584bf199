// Eviction from the pools by gathered attention weight, and slots for the chunks to come.
//
// A (request, KV head) unit u owns slots u S .. u S + S - 1 of the pool.  With n0 = ceil(kv_len / cs)
// chunks so far and n1 = ceil((kv_len + new_len) / cs) to be, R chunks resident and N of n0 .. n1 - 1
// without a slot, E = clamp(R + N - keep, 0, candidates) chunks leave: those of the smallest weight among the
// resident chunks c with first <= c < n0 - last, the lower chunk first where weights are equal.
// The N new chunks then take free slots, ascending both.
//
// One CTA a unit, two an SM.  A radix select over the weights' order keys (a NaN below every number, -0 as +0) in
// digits of 11 bits finds the E-th smallest: 2,048 bins spread exponents over banks, and the first two digits
// leave one or two keys, or equal ones, so a third is rarely looked at.  What bounds it is the chain of
// passes and barriers, not its bytes.
//   k_evict       up to 8,192 chunks: a lane keeps up to 16 of them in registers (slot, key), read once, all
//                 loads on their way together; ranks are ballots, so every access is a whole line
//   k_evict_many  more: 512 threads cannot hold them, and 1,024 leave room for one CTA an SM.  The residents
//                 become entries (key, chunk, slot) in shared memory, in any order; chunk order is kept in bitmaps
//                 with a prefix of each word, so a rank is a prefix and a population count
// 512 units of 16,384, 12,288, 8,192, 4,096 chunks, a quarter resident: k_evict_many 61, 51, 41, 33 us, k_evict 93, 84 (1,024
// threads), 43, 27; 32 units: 22, 19, 16, 14 and 22, 21, 16, 11.
#include "dd_pages.cuh"

namespace dd {

namespace {

enum : uint32_t { kAbsent = 0, kStays = 1, kMay = 2, kNew = 3 };
constexpr int kDigit = 11, kBins = 1 << kDigit;

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// An error that was pending before the launch stops all of its units, one that a unit of the launch reports no
// other: `raised` is the number of the last launch that has reported one, and a unit's count of launches is the
// number of this one (every launch runs every unit).  One thread a CTA; the others take its answer behind a barrier.
struct Launch {
  uint32_t number;
  bool stopped;
};
__device__ __forceinline__ Launch begin_launch(const EvictArgs &a, int u) {
  Launch l;
  const int32_t status = load_status(a.status);
  l.number = a.launches[u] + 1u;
  a.launches[u] = l.number;
  l.stopped = false;
  if (status != 0) {
    __threadfence();                                         // (whoever set the word has written its launch before)
    l.stopped = *reinterpret_cast<const volatile uint32_t *>(a.raised) != l.number;
  }
  return l;
}

__device__ __forceinline__ void report(const EvictArgs &a, uint32_t launch, int32_t code) {
  *reinterpret_cast<volatile uint32_t *>(a.raised) = launch;
  __threadfence();
  set_status(a.status, code);
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

template <int N>
__global__ void __launch_bounds__(512, 2) k_evict(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  const int words = (a.S + 31) / 32;
  uint32_t *hist = sm;                                       // [kBins]
  uint32_t *used = sm + kBins;                               // [words] slots held
  uint16_t *free_slot = reinterpret_cast<uint16_t *>(used + words), *owner = free_slot + a.S;   // [S] each
  __shared__ int scratch[3][33];
  __shared__ int s_bad, s_stopped;
  __shared__ uint32_t s_digit, s_rank, s_count, s_low, s_high;

  pdl_wait();
  pdl_trigger();
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int b = u / a.Hkv;
  const int64_t row = (int64_t)u * a.C, base = (int64_t)u * a.S;
  const int c0 = warp * 32 * N + lane;
  const uint32_t below = (1u << lane) - 1u;
  const int32_t *const slots = a.resident_slot + row + c0;
  const float *const weights = a.weight + row + c0;
  int32_t slot[N];
  uint32_t key[N], state = 0u;                               // state: two bits a chunk
#pragma unroll
  for (int k = 0; k < N; ++k) slot[k] = c0 + 32 * k < a.C ? slots[32 * k] : -1;
#pragma unroll
  for (int k = 0; k < N; ++k) key[k] = c0 + 32 * k < a.C ? __float_as_uint(weights[32 * k]) : 0u;
  const int kv = a.kv_len[b], more = a.new_len ? a.new_len[b] : 0;
  uint32_t launch = 0u;                                      // (thread 0's, which reports)
  if (tid == 0) {
    const Launch l = begin_launch(a, u);
    launch = l.number, s_stopped = l.stopped;
  }
  bool bad = kv < 0 || more < 0 || (int64_t)kv + more > (int64_t)a.C * a.cs;
  const int n0 = bad ? 0 : (kv + a.cs - 1) / a.cs, n1 = bad ? 0 : (kv + more + a.cs - 1) / a.cs;

  if (tid == 0) s_bad = 0, s_low = 0xFFFFFFFFu, s_high = 0u, s_count = 0u;
  for (int i = tid; i < words; i += blockDim.x) used[i] = 0u;
  __syncthreads();
  if (s_stopped) return;
  Counts n = {0, 0, 0};                                      // resident, new, candidates
  const int may0 = a.first, may1 = n0 - a.last;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = c0 + 32 * k;
    if (slot[k] >= 0) {
      // a slot of another unit, or of two chunks
      const int64_t s = slot[k] - base;
      bool ok = s >= 0 && s < a.S;
      if (ok) ok = (atomicOr(&used[(int)s >> 5], 1u << (s & 31)) >> (s & 31) & 1u) == 0u;
      if (!ok) s_bad = 1;
      const bool may = c >= may0 && c < may1;
      state |= (may ? kMay : kStays) << (2 * k);
      n.a += 1, n.c += may;
    } else if (c >= n0 && c < n1 && c < a.C) {
      state |= kNew << (2 * k);
      n.b += 1;
    }
    key[k] = order_key(__uint_as_float(key[k]));
  }
  n.a = __reduce_add_sync(0xffffffffu, n.a), n.b = __reduce_add_sync(0xffffffffu, n.b), n.c = __reduce_add_sync(0xffffffffu, n.c);
  Counts all;
  warp_prefix(n, scratch, all, warp, lane, warps);
  bad = bad || s_bad != 0;
  if (bad) {
    // left as it was
    if (tid == 0) {
      report(a, launch, DD_ERR_DEVICE_CHECK);
      if (a.evicted_cnt) a.evicted_cnt[u] = 0;
      if (a.list_cnt) a.list_cnt[u] = 0;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (c0 + 32 * k < a.C) a.resident_out[row + c0 + 32 * k] = slot[k];
    return;
  }
  const int leave = min(max(all.a + all.b - a.keep, 0), all.c);

  // the digits of the leave-th smallest key, from the top, until all keys that share them leave
  int shift = 32;
  uint32_t bound = 0u, rank = (uint32_t)leave;               // of those that share the digits found so far
  uint32_t shared = (uint32_t)all.c;                         // how many share them
  bool ties = leave > 0;
  for (int width = kDigit; ties && shift > 0; ) {
    const int next = max(0, shift - width);
    for (int i = tid; i < kBins; i += blockDim.x) hist[i] = 0u;
    __syncthreads();
    const uint32_t mask = (1u << (shift - next)) - 1u;
    uint32_t low = 0xFFFFFFFFu, high = 0u;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if ((state >> (2 * k) & 3u) == kMay && (shift == 32 || key[k] >> shift == bound)) {
        atomicAdd(&hist[key[k] >> next & mask], 1u);
        low = min(low, key[k]), high = max(high, key[k]);
      }
    low = __reduce_min_sync(0xffffffffu, low), high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0 && low <= high) atomicMin(&s_low, low), atomicMax(&s_high, high);
    __syncthreads();
    if (s_low == s_high) {
      // all alike (chunks that nothing has looked at): no digit tells them apart
      bound = s_low, shift = 0, ties = shared != rank;
      break;
    }
    const int per = kBins / (int)blockDim.x, from = tid * per;   // (128, 256 or 512 threads)
    int sum = 0;
    for (int i = 0; i < per; ++i) sum += (int)hist[from + i];
    Counts t, mine = {0, 0, 0};
    const int incl = warp_incl_scan(sum);
    mine.a = __shfl_sync(0xffffffffu, incl, 31);
    uint32_t before = (uint32_t)(warp_prefix(mine, scratch, t, warp, lane, warps).a + incl - sum);
    if (before < rank && rank <= before + (uint32_t)sum)
      for (int i = 0; i < per; ++i) {
        const uint32_t v = hist[from + i];
        if (before < rank && rank <= before + v) s_digit = from + i, s_rank = rank - before, s_count = v;
        before += v;
      }
    __syncthreads();
    bound = shift == 32 ? s_digit : bound << (shift - next) | s_digit;
    rank = s_rank, shared = s_count, ties = shared != rank, shift = next;
    if (tid == 0) s_low = 0xFFFFFFFFu, s_high = 0u;        // (read before the barrier in front of this)
  }

  // the first `rank` of the keys that share the digits leave, in chunk order
  Counts m = {0, 0, 0};
  if (ties)
#pragma unroll
    for (int k = 0; k < N; ++k)
      m.a += __popc(__ballot_sync(0xffffffffu, (state >> (2 * k) & 3u) == kMay && key[k] >> shift == bound));
  int tied = ties ? warp_prefix(m, scratch, all, warp, lane, warps).a : 0;
  m = {0, 0, 0};                                             // leaving, new, staying
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t st = state >> (2 * k) & 3u;
    bool go = false;
    if (leave > 0) {
      const uint32_t top = key[k] >> shift;
      go = st == kMay && top <= bound;
      if (ties) {
        const bool tie = st == kMay && top == bound;
        const uint32_t in = __ballot_sync(0xffffffffu, tie);
        if (tie) go = tied + __popc(in & below) < (int)rank;
        tied += __popc(in);
      }
    }
    // (from here on: kMay leaves)
    if (go) {
      const int s = (int)(slot[k] - base);
      atomicAnd(&used[s >> 5], ~(1u << (s & 31)));
    } else if (st == kMay) {
      state ^= (kMay ^ kStays) << (2 * k);
    }
    m.a += go, m.b += st == kNew, m.c += st == kStays || (st == kMay && !go);
  }
  m.a = __reduce_add_sync(0xffffffffu, m.a), m.b = __reduce_add_sync(0xffffffffu, m.b), m.c = __reduce_add_sync(0xffffffffu, m.c);
  const Counts pre = warp_prefix(m, scratch, all, warp, lane, warps);

  // the free slots, ascending: a thread a word of 32
  int n_free = 0;
  {
    uint32_t w = 0u;
    if (tid < words) {
      w = ~used[tid];
      if (tid == words - 1 && (a.S & 31)) w &= (1u << (a.S & 31)) - 1u;
    }
    const int f = __popc(w), incl = warp_incl_scan(f);
    Counts t, fc = {__shfl_sync(0xffffffffu, incl, 31), 0, 0};
    int at = warp_prefix(fc, scratch, t, warp, lane, warps).a + incl - f;
    n_free = t.a;
    while (w) {
      const int bit = __ffs((int)w) - 1;
      w &= w - 1;
      if (at < all.b) free_slot[at] = (uint16_t)(32 * tid + bit);
      ++at;
    }
    for (int i = tid; i < a.S; i += blockDim.x) owner[i] = 0xFFFFu;
  }
  __syncthreads();
  if (all.b > n_free && tid == 0) report(a, launch, DD_ERR_CAPACITY);
  const int given = min(all.b, n_free);

  // (new chunks lie behind n0, among the residents there)
  int gone = pre.a, listed = pre.c + min(pre.b, given), fresh = pre.b;
  int32_t *const out = a.resident_out + row + c0;
  int32_t *const idx_to = a.list_idx ? a.list_idx + (int64_t)u * a.umax : nullptr;
  int32_t *const slot_to = a.list_slot + (a.list_idx ? (int64_t)u * a.umax : 0);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = c0 + 32 * k;
    const uint32_t st = state >> (2 * k) & 3u;
    int32_t now = st == kStays ? slot[k] : -1;
    if (all.b > 0) {
      const uint32_t in_new = __ballot_sync(0xffffffffu, st == kNew);
      const int my_new = fresh + __popc(in_new & below);
      if (st == kNew && my_new < given) {
        now = (int32_t)base + free_slot[my_new];
        if (a.last_used) a.last_used[now] = a.step;
      }
      fresh += __popc(in_new);
    }
    if (c < a.C) out[32 * k] = now;
    const uint32_t in = __ballot_sync(0xffffffffu, now >= 0);
    if (now >= 0) {
      owner[now - base] = (uint16_t)c;
      const int at = listed + __popc(in & below);
      if (idx_to) idx_to[at] = c, slot_to[at] = now;
    }
    listed += __popc(in);
    if (a.evicted) {
      const uint32_t in_go = __ballot_sync(0xffffffffu, st == kMay);
      if (st == kMay) a.evicted[base + gone + __popc(in_go & below)] = c;
      gone += __popc(in_go);
    }
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

constexpr uint32_t kLeaves = 0x8000u;   // of an entry's chunk: it may leave

// Exclusive prefix over the block's threads, and the total.  `scratch` holds 33 ints; two barriers, none at the end.
__device__ __forceinline__ int block_prefix(int v, int *scratch, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int incl = warp_incl_scan(v);
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int x = lane < warps ? scratch[lane] : 0, s = warp_incl_scan(x);
    __syncwarp();
    scratch[lane] = s - x;
    if (lane == 31) scratch[32] = s;
  }
  __syncthreads();
  *total = scratch[32];
  return scratch[warp] + incl - v;
}

// The rank of bit c among a bitmap's, whose words have the prefix `pre`.
__device__ __forceinline__ int rank_of(const uint32_t *bits, const uint16_t *pre, int c) {
  return pre[c >> 5] + __popc(bits[c >> 5] & ((1u << (c & 31)) - 1u));
}

struct EvictSmem {
  uint32_t *hist, *used, *here, *gone, *tied, *key;   // bins; bitmaps of slots and chunks; entries' keys [S]
  uint16_t *pre, *chunk, *slot, *owner, *spare;       // words' prefix; entries [S]; chunk of a slot, free slots [S]
};

__host__ __device__ inline size_t evict_smem(int C, int S, uint32_t *w, EvictSmem *m) {
  const int cw = (C + 31) / 32, sw = (S + 31) / 32;
  EvictSmem x;
  x.hist = w, x.used = x.hist + kBins, x.here = x.used + sw, x.gone = x.here + cw, x.tied = x.gone + cw, x.key = x.tied + cw;
  x.pre = reinterpret_cast<uint16_t *>(x.key + S);
  x.chunk = x.pre + cw, x.slot = x.chunk + S, x.owner = x.slot + S, x.spare = x.owner + S;
  if (m) *m = x;
  return (size_t)(kBins + sw + 3 * cw + S) * 4 + (size_t)(cw + 4 * S) * 2;
}

__global__ void __launch_bounds__(512, 2) k_evict_many(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ int scratch[2][33], s_bad, s_stopped, s_entries, s_may;
  __shared__ uint32_t s_digit, s_rank, s_count, s_low, s_high;
  constexpr int N = 8;                                       // chunks of a lane at a time (16: 66 us for 61, 4: 64)
  EvictSmem m;
  evict_smem(a.C, a.S, sm, &m);
  const int cw = (a.C + 31) / 32, sw = (a.S + 31) / 32;

  pdl_wait();
  pdl_trigger();
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int b = u / a.Hkv;
  const int64_t row = (int64_t)u * a.C, base = (int64_t)u * a.S;
  const uint32_t below = (1u << lane) - 1u;
  int32_t *const out = a.resident_out + row;
  const bool copy = a.resident_out != a.resident_slot;
  int32_t slot[N];
  float weight[N];
  auto load = [&](int c0) {
#pragma unroll
    for (int k = 0; k < N; ++k) slot[k] = c0 + 32 * k < a.C ? a.resident_slot[row + c0 + 32 * k] : -1;
#pragma unroll
    for (int k = 0; k < N; ++k) weight[k] = c0 + 32 * k < a.C ? a.weight[row + c0 + 32 * k] : 0.f;
  };
  int c0 = warp * 32 * N + lane;
  load(c0);
  const int kv = a.kv_len[b], more = a.new_len ? a.new_len[b] : 0;
  uint32_t launch = 0u;                                      // (thread 0's, which reports)
  if (tid == 0) {
    const Launch l = begin_launch(a, u);
    launch = l.number, s_stopped = l.stopped;
  }
  bool bad = kv < 0 || more < 0 || (int64_t)kv + more > (int64_t)a.C * a.cs;
  const int n0 = bad ? 0 : (kv + a.cs - 1) / a.cs, n1 = bad ? 0 : (kv + more + a.cs - 1) / a.cs;

  if (tid == 0) s_bad = 0, s_entries = 0, s_may = 0, s_low = 0xFFFFFFFFu, s_high = 0u;
  for (int i = tid; i < sw + 3 * cw; i += nt) m.used[i] = 0u;      // (and the bitmaps of chunks behind it)
  __syncthreads();
  if (s_stopped) return;
  const int may0 = a.first, may1 = n0 - a.last;
  const uint32_t slots = base <= INT_MAX ? (uint32_t)a.S : 0u;     // (a unit behind all 32-bit slots has none)
  int mays = 0;
  for (;;) {
    uint32_t in[N];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) in[k] = __ballot_sync(0xffffffffu, slot[k] >= 0), mine += __popc(in[k]);
    int first = 0;                                             // one place for all of a warp's entries
    if (lane == 0 && mine) first = atomicAdd(&s_entries, mine);
    first = __shfl_sync(0xffffffffu, first, 0);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = c0 + 32 * k;
      if (copy && c < a.C) out[c] = slot[k];                   // as it was, until it turns out otherwise
      if (lane == 0 && in[k]) m.here[c >> 5] = in[k];
      if (slot[k] >= 0) {
        // a slot of another unit, or more chunks than slots (two chunks of a slot: see below)
        const uint32_t s = (uint32_t)slot[k] - (uint32_t)base;
        const int at = first + __popc(in[k] & below);
        if (s >= slots || at >= a.S) {
          s_bad = 1;
        } else {
          atomicOr(&m.used[s >> 5], 1u << (s & 31));
          const bool may = c >= may0 && c < may1;
          mays += may;
          m.key[at] = order_key(weight[k]);
          m.chunk[at] = (uint16_t)(may ? c | kLeaves : c), m.slot[at] = (uint16_t)s;
        }
      }
      first += __popc(in[k]);
    }
    // (a warp's next chunks begin at c0 - lane)
    c0 += nt * N;
    if (c0 - lane >= a.C) break;
    load(c0);
  }
  mays = __reduce_add_sync(0xffffffffu, mays);
  if (lane == 0 && mays) atomicAdd(&s_may, mays);
  __syncthreads();
  // the new chunks: a thread a word
  uint32_t fresh = 0u;
  if (tid < cw) {
    const int lo = min(max(n0 - 32 * tid, 0), 32), hi = min(max(n1 - 32 * tid, 0), 32);
    const uint32_t range = (hi == 32 ? ~0u : (1u << hi) - 1u) & ~(lo == 32 ? ~0u : (1u << lo) - 1u);
    fresh = ~m.here[tid] & range;
  }
  // (and how many slots are held: as many as chunks hold one)
  int both;
  const int my_new = block_prefix(__popc(fresh) | __popc(tid < sw ? m.used[tid] : 0u) << 16, scratch[0], &both) & 0xFFFF;
  const int n_new = both & 0xFFFF, entries = s_entries;
  bad = bad || s_bad != 0 || both >> 16 != entries;
  if (bad) {
    // left as it was
    if (tid == 0) {
      report(a, launch, DD_ERR_DEVICE_CHECK);
      if (a.evicted_cnt) a.evicted_cnt[u] = 0;
      if (a.list_cnt) a.list_cnt[u] = 0;
    }
    return;
  }
  const int leave = min(max(entries + n_new - a.keep, 0), s_may);

  // the digits of the leave-th smallest key, from the top, until all keys that share them leave
  int shift = 32;
  uint32_t bound = 0u, rank = (uint32_t)leave;               // of those that share the digits found so far
  uint32_t shared = (uint32_t)s_may;                         // how many share them
  bool ties = leave > 0;
  while (ties && shift > 0) {
    const int next = max(0, shift - kDigit);
    for (int i = tid; i < kBins; i += nt) m.hist[i] = 0u;
    __syncthreads();
    const uint32_t mask = (1u << (shift - next)) - 1u;
    uint32_t low = 0xFFFFFFFFu, high = 0u;
    for (int i = tid; i < entries; i += nt) {
      const uint32_t k = m.key[i];
      if ((m.chunk[i] & kLeaves) && (shift == 32 || k >> shift == bound)) {
        atomicAdd(&m.hist[k >> next & mask], 1u);
        low = min(low, k), high = max(high, k);
      }
    }
    low = __reduce_min_sync(0xffffffffu, low), high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0 && low <= high) atomicMin(&s_low, low), atomicMax(&s_high, high);
    __syncthreads();
    if (s_low == s_high) {
      // all alike (chunks that nothing has looked at): no digit tells them apart
      bound = s_low, shift = 0, ties = shared != rank;
      break;
    }
    const int per = kBins / nt, from = tid * per;
    int sum = 0, all;
    for (int i = 0; i < per; ++i) sum += (int)m.hist[from + i];
    uint32_t before = (uint32_t)block_prefix(sum, scratch[1], &all);
    if (before < rank && rank <= before + (uint32_t)sum)
      for (int i = 0; i < per; ++i) {
        const uint32_t v = m.hist[from + i];
        if (before < rank && rank <= before + v) s_digit = from + i, s_rank = rank - before, s_count = v;
        before += v;
      }
    __syncthreads();
    bound = shift == 32 ? s_digit : bound << (shift - next) | s_digit;
    rank = s_rank, shared = s_count, ties = shared != rank, shift = next;
    if (tid == 0) s_low = 0xFFFFFFFFu, s_high = 0u;          // (read before the barriers in front of this)
  }

  int total;
  if (ties) {
    // of the keys that share the digits the first `rank` leave, in chunk order
    for (int i = tid; i < entries; i += nt) {
      const int c = m.chunk[i] & (kLeaves - 1u);
      if ((m.chunk[i] & kLeaves) && m.key[i] >> shift == bound) atomicOr(&m.tied[c >> 5], 1u << (c & 31));
    }
    __syncthreads();
    const int before = block_prefix(tid < cw ? __popc(m.tied[tid]) : 0, scratch[0], &total);
    if (tid < cw) m.pre[tid] = (uint16_t)before;
    __syncthreads();
  }
  if (leave > 0)
    for (int i = tid; i < entries; i += nt) {
      const uint32_t chunk = m.chunk[i], top = m.key[i] >> shift;
      const int c = (int)(chunk & (kLeaves - 1u));
      if ((chunk & kLeaves) && (top < bound || (top == bound && (!ties || rank_of(m.tied, m.pre, c) < (int)rank)))) {
        const int s = m.slot[i];
        atomicAnd(&m.used[s >> 5], ~(1u << (s & 31)));
        atomicAnd(&m.here[c >> 5], ~(1u << (c & 31)));
        atomicOr(&m.gone[c >> 5], 1u << (c & 31));
        out[c] = -1;
      }
    }
  for (int i = tid; i < a.S; i += nt) m.owner[i] = 0xFFFFu;
  __syncthreads();

  // the free slots, ascending, as many as are needed: a thread a word
  int n_free;
  {
    uint32_t w = 0u;
    if (tid < sw) {
      w = ~m.used[tid];
      if (tid == sw - 1 && (a.S & 31)) w &= (1u << (a.S & 31)) - 1u;
    }
    int at = block_prefix(__popc(w), scratch[1], &n_free);
    for (; w && at < n_new; w &= w - 1, ++at) m.spare[at] = (uint16_t)(32 * tid + __ffs((int)w) - 1);
  }
  __syncthreads();
  if (n_new > n_free && tid == 0) report(a, launch, DD_ERR_CAPACITY);
  const int given = min(n_new, n_free);
  // (a word has one thread: no other writes it now)
  uint32_t placed = 0u;
  int j = my_new;
  for (uint32_t w = fresh; w && j < given; w &= w - 1, ++j) {
    const int c = 32 * tid + __ffs((int)w) - 1, s = m.spare[j];
    placed |= w & (0u - w);
    out[c] = (int32_t)base + s;
    m.owner[s] = (uint16_t)c;
    if (a.last_used) a.last_used[base + s] = a.step;
  }
  if (placed) m.here[tid] |= placed;
  // the chunks that are resident now, by word
  {
    const int before = block_prefix(tid < cw ? __popc(m.here[tid]) : 0, scratch[0], &total);
    if (tid < cw) m.pre[tid] = (uint16_t)before;
  }
  __syncthreads();
  int32_t *const idx_to = a.list_idx ? a.list_idx + (int64_t)u * a.umax : nullptr;
  int32_t *const slot_to = a.list_slot + (a.list_idx ? (int64_t)u * a.umax : 0);
  for (int i = tid; i < entries; i += nt) {
    const int c = m.chunk[i] & (kLeaves - 1u), s = m.slot[i];
    if (!(m.here[c >> 5] >> (c & 31) & 1u)) continue;
    m.owner[s] = (uint16_t)c;
    if (idx_to) {
      const int at = rank_of(m.here, m.pre, c);
      idx_to[at] = c, slot_to[at] = (int32_t)base + s;
    }
  }
  if (idx_to) {
    j = my_new;
    for (uint32_t w = placed; w; w &= w - 1, ++j) {
      const int c = 32 * tid + __ffs((int)w) - 1, at = rank_of(m.here, m.pre, c);
      idx_to[at] = c, slot_to[at] = (int32_t)base + m.spare[j];
    }
  }
  if (a.evicted && leave > 0) {
    // the chunks that left (nothing ties any more: their words' prefix takes that place)
    uint16_t *const gone_pre = reinterpret_cast<uint16_t *>(m.tied);
    const int before = block_prefix(tid < cw ? __popc(m.gone[tid]) : 0, scratch[1], &n_free);
    if (tid < cw) gone_pre[tid] = (uint16_t)before;
    __syncthreads();
    for (int i = tid; i < entries; i += nt) {
      const int c = m.chunk[i] & (kLeaves - 1u);
      if (m.gone[c >> 5] >> (c & 31) & 1u) a.evicted[base + rank_of(m.gone, gone_pre, c)] = c;
    }
  }
  if (tid == 0) {
    if (a.evicted_cnt) a.evicted_cnt[u] = leave;
    if (a.list_cnt) a.list_cnt[u] = total;
  }
  __syncthreads();
  if (a.slot_chunk || a.last_used)
    for (int i = tid; i < a.S; i += nt) {
      const uint16_t c = m.owner[i];
      if (a.slot_chunk) a.slot_chunk[base + i] = c == 0xFFFFu ? -1 : (int32_t)c;
      if (a.last_used && c == 0xFFFFu) a.last_used[base + i] = -1;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s) {
  const int lines = (a.C + 31) / 32, words = (a.S + 31) / 32;
  if (lines > 256) {
    // (16,384 chunks and slots at most: 512 words of a bitmap, one a thread)
    const size_t smem = evict_smem(a.C, a.S, nullptr, nullptr);
    const cudaError_t e = set_dyn_smem((const void *)k_evict_many, smem);
    return e != cudaSuccess ? e : launch_k(k_evict_many, dim3(a.units), dim3(512), smem, s, a);
  }
  // 16 warps at most (two CTAs an SM: 2,048 chunks of 256 units 9.9 us; 18.1 with 32 warps, in two rounds), four
  // at least, and a thread for each word of the slots' bitmap
  int n = 1;
  while (n < 16 && n * 16 < lines) n *= 2;
  int warps = (lines + n - 1) / n;
  if (warps < 4) warps = 4;
  if (32 * warps < words) warps = (words + 31) / 32;
  // (the bins are shared out evenly among a power of two of threads)
  int pow = 4;
  while (pow < warps) pow *= 2;
  const size_t smem = (size_t)(kBins + words) * 4 + (size_t)a.S * 4;
  auto go = [&](auto *kernel) {
    const cudaError_t e = set_dyn_smem((const void *)kernel, smem);
    return e != cudaSuccess ? e : launch_k(kernel, dim3(a.units), dim3(32 * pow), smem, s, a);
  };
  switch (n) {
    case 1: return go(&k_evict<1>);
    case 2: return go(&k_evict<2>);
    case 4: return go(&k_evict<4>);
    case 8: return go(&k_evict<8>);
    default: return go(&k_evict<16>);
  }
}

}  // namespace dd
