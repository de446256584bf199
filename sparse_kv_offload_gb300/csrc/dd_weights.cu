// The attention weight that each listed chunk has gathered from new tokens:
//   weight[b,g,c] = decay * weight[b,g,c] + sum over tokens t, heads h of KV head g, rows i of
//                   chunk c that t sees:  exp(scale q_{t,h}.k_i - lse_{t,h}),
// lse as the attention of these tokens has left it.  One product and one exponential a pair, no
// second product: half of the attention's operations, and K read once.
//
// The product is turned round, S = K Q^T with 128 keys on the rows of tensor memory, so that a
// thread owns a key and its sum over the query rows stays in a register; only a chunk's rows
// are added up across lanes.  With queries on the rows every tile would need 128 column sums.
// Sums are fp32, in an order that depends on the sizes alone (no atomics on values).
//   warps 0-3, 4-7  exponentials and sums of a pair's two tiles of 128 keys
//   warp 8          the products, two of each tile on the way in tensor memory
//   warp 9          hands out the work and brings a third of a pair's keys, as warps 10 and 11 do (two or
//                   three pairs on the way; a warp issues a box in some 100 cycles, and chunks of 16 rows are 32 boxes a pair)
//   warp 11         Q's tiles (three on the way) and their log-sum-exps, too
//
// With few query rows (one tile) the keys stream past the queries, an equal slice of all pairs a CTA; with many, the
// queries stream past a pair.  Where the pairs alone would leave CTAs idle the rows are cut too, and
// a pair's parts (16 sums at most) are added up in order by whoever finishes last.
//
// What bounds it: with many query rows no pipe, but what two warps a scheduler can have on the way: a load out of tensor
// memory, multiply-adds, exponentials and additions follow one another (2 requests, 2,048 tokens, 64 heads, 16K of
// context: 1.03 ms, 12.4 scores a clock and SM of the 32 exponentials that ex2.approx alone runs at; XU and tensor pipe 42%
// each on a smaller case; a quarter of the exponentials as polynomials on the FMA pipe cost 19%).  With two tiles of
// query rows a pair its ends count as well (last 32 tokens of 8 prompts, 64 heads: 98 to 123 us by lengths, 11.2 a clock).
// With one token a request HBM (16 whole caches of up to 32K in chunks of 16: 111 to 126 us by lengths, 6,300 GB/s;
// 3% more with two pairs on the way, 50% as items, 15% with a list's entries looked at right behind their loads).
#include "dd_pages.cuh"

namespace dd {

namespace {

constexpr int kSums = 8;                             // warps of exponentials and sums
constexpr int kThreads = (kSums + 4) * 32;
constexpr int kQ = 3;                                // tiles of queries on the way
constexpr int kPairs = 3;                            // pairs of tiles of keys on the way, two with many query rows
constexpr int kRec = 4;                              // records of pairs
constexpr uint32_t kTmem = 512;                      // S: two of 128 columns for each tile of a pair
constexpr int kItemsPerCta = 8;

struct Pair {
  int unit, start, len;
  int last;                   // position of the last token, -1 where there is none
  int tok0;                   // the first token that counts
  int r0, r1;                 // tiles of query rows to go through
  int keep_q;                 // one tile of queries for all pairs of the item: 1 first, 2 last, 3 both, 4 neither, 0 no
  int parts, part0, part, cut;   // ranges of rows, slots, arrival counter
  int slot[16];               // of its chunks
  int pos[16];                // positions of the first rows of its chunks, INT_MAX where there is none
};

struct Misc {
  uint64_t bars[40];
  Pair pair[kRec];
  alignas(16) float lse[kQ][128];   // times -log2 e; -inf where there is no row
  float sum[2][2][4];                // [buffer][stream][32 rows], for chunks of 64
  long long work[kThreads / 32];      // units' pairs by rows of each warp, their pairs, and of the first blocks of 32 units
  int pairs[kThreads / 32], one[kThreads / 32], block[32];
  int dead, pending;
  uint32_t tmem;
};

constexpr size_t kTiles = (size_t)7 * kTileBytes;    // kQ tiles of queries and 2 pairs, or kQ of 32 rows and 3 pairs
static_assert(kQ * 2 * 32 * 128 + kPairs * 2 * kTileBytes <= kTiles, "few query rows");
constexpr size_t kSmem = kTiles + sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory of a CTA");

struct WeightsParams {
  CUtensorMap q, k, kst;
  PagesArgs a;
  const float *lse;
  float *weight;
  int window;
  float decay;
  float *parts;               // [slots][16]
  WorkCounters w;
};

struct Unit {
  int cnt, start, len, tok0, pairs, rows;     // pairs of tiles of keys, tiles of query rows
};

__device__ __forceinline__ Unit load_unit(const WeightsParams &p, int u) {
  Unit r;
  const Request q = load_request(p.a, u / p.a.Hkv);
  r.cnt = load_count(p.a, u);
  r.start = q.start, r.len = q.len;
  r.tok0 = p.window > 0 ? max(0, q.len - p.window) : 0;
  r.pairs = ceil_div(r.cnt * p.a.cs, 2 * kTileKeys);
  r.rows = max(1, ceil_div(q.len - r.tok0, p.a.tt));       // (without tokens the weights still decay)
  return r;
}

// Tiles of query rows of an item.  With P CTAs: pairs whose rows are cut <= 8 P, items of those <= 16 P.
__device__ __forceinline__ int rows_cut_of(long long pairs, long long work, bool one, int cta) {
  const long long most = (long long)kItemsPerCta * cta;
  return one || pairs >= most ? INT_MAX : (int)max(1ll, (work + most - 1) / most);
}

__global__ void __launch_bounds__(kThreads, 1) k_weights(const __grid_constant__ WeightsParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc &x = *reinterpret_cast<Misc *>(smem + kTiles);
  const PagesArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rows_tile = a.tt * a.G, chunks = kTileKeys / a.cs;
  const bool few = rows_tile <= 32;
  const uint32_t q_half = few ? 32 * 128 : kTileHalfBytes, kPair = few ? kPairs : 2;
  const uint32_t q0 = smem_u32(smem), k0 = q0 + kQ * 2 * q_half;
  const uint32_t bars = smem_u32(x.bars);
  const uint32_t rec_full = bars, pair_full = rec_full + 8 * kRec, pair_free = pair_full + 8 * kRec, k_free = pair_free + 8 * kRec,
                 q_full = k_free + 8 * kPairs, q_free = q_full + 8 * kQ, s_full = q_free + 8 * kQ, s_free = s_full + 32,
                 mma_done = s_free + 32, summed = mma_done + 8;
  if (tid == 0) {
    // a pair: its record and its tiles; free again after the products (tiles) and the sums (record)
    for (int i = 0; i < kRec; ++i)
      mbar_init(rec_full + 8 * i, 1), mbar_init(pair_full + 8 * i, 1), mbar_init(pair_free + 8 * i, kSums + 3);
    for (int i = 0; i < kPairs; ++i) mbar_init(k_free + 8 * i, 1);
    // a tile of queries: its copy and its log-sum-exps; free after the products and the sums
    for (int i = 0; i < kQ; ++i) mbar_init(q_full + 8 * i, 1), mbar_init(q_free + 8 * i, kSums + 1);
    for (int i = 0; i < 4; ++i) mbar_init(s_full + 8 * i, 2), mbar_init(s_free + 8 * i, 4);
    mbar_init(mma_done, 1), mbar_init(summed, 4), mbar_init(summed + 8, 4);
    x.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSums) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&x.tmem)), "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // query rows behind a tile's last are never written: zeros once
  const int blank = (few ? 32 : 128) - rows_tile;
  for (int e = tid; e < kQ * 2 * blank * 8; e += kThreads)
    *reinterpret_cast<uint4 *>(smem + e / (blank * 8) * q_half + rows_tile * 128 + e % (blank * 8) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_fence_before();
  pdl_wait();
  pdl_trigger();
  if (tid == 0) x.pending = load_status(a.status);
  // what there is to do: a warp's blocks of 32 units each
  const int units = a.B * a.Hkv;
  {
    int pairs = 0, one = 1;
    long long work = 0;
    for (int u0 = 32 * warp; u0 < units; u0 += kThreads) {
      Unit r = {0, 0, 0, 0, 0, 1};
      if (u0 + lane < units) r = load_unit(p, u0 + lane);
      const int sum = __reduce_add_sync(0xffffffffu, r.pairs);
      if (lane == 0 && u0 < 1024) x.block[u0 >> 5] = sum;
      pairs += sum, work += (long long)r.pairs * r.rows, one &= r.rows == 1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
    one = __all_sync(0xffffffffu, one);
    if (lane == 0) x.pairs[warp] = pairs, x.work[warp] = work, x.one[warp] = one;
  }
  __syncthreads();
  tc_fence_after();
  const bool pending = x.pending != 0;
  const uint32_t tmem = x.tmem;

  auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_or_dead(bar, parity, &x.dead, a.raised));
  };
  // whether a step of a pair takes a new tile of queries, and whether it is the tile's last
  auto new_q = [](int keep) { return keep == 0 || (keep & 1); };
  auto last_q = [](int keep) { return keep == 0 || keep == 2 || keep == 3; };
  // a third of a pair's 2 * chunks chunks: a lane brings half of the columns of one (its slot and position in the
  // lane of the chunk's number; zeros for one behind the last token's position)
  auto load_third = [&](int third, int slot, int pos, int last, uint32_t st, uint32_t bar) {
    const int lo = 2 * chunks * third / 3, hi = 2 * chunks * (third + 1) / 3, ch = min(lo + (lane >> 1), 31);
    const int sl = __shfl_sync(0xffffffffu, slot, ch), at = __shfl_sync(0xffffffffu, pos, ch);
    if (ch < hi) load_chunk(p.k, p.kst, a, sl, at > last ? INT_MAX : at, lane & 1, k0 + (st * 2 + ch / chunks) * kTileBytes + ch % chunks * a.cs * 128, bar);
  };
  if (pending) {
    // no work; the counters below are left all the same
  } else if (warp == kSums + 1) {
    // ------------------------------------------------------- the work, and K's tiles
    const int cta = (int)gridDim.x, part_of = min(lane, kThreads / 32 - 1);
    const bool some = lane < kThreads / 32;
    const int pairs = __reduce_add_sync(0xffffffffu, some ? x.pairs[part_of] : 0);
    const bool one = __all_sync(0xffffffffu, x.one[part_of]);
    long long work = some ? x.work[part_of] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
    const int rows_cut = rows_cut_of(pairs, work, one, cta);
    const int64_t staged = staged_slots(a);

    // One tile of query rows a unit: every CTA has an equal slice of all units' pairs, laid end to end.  Else
    // items, a pair by a range of rows each, are handed out by tickets, the first by number.
    const int per_cta = (int)((pairs + cta - 1) / cta);
    int base_u = -32, items_before = 0, items_here = 0, cuts_before = 0, cuts_here = 0, parts_before = 0, parts_here = 0;
    Unit mine = {0, 0, 0, 0, 0, 0};
    int ranges = 0, items = 0, items_pre = 0, cuts_pre = 0, parts_pre = 0;
    int want = one ? (int)blockIdx.x * per_cta : (int)blockIdx.x;
    const int slice_end = want + per_cta;
    if (one && units <= 1024) {
      // the block of units that the slice begins in
      const int incl = warp_incl_scan(32 * lane < units ? x.block[lane] : 0);
      const uint32_t past = __ballot_sync(0xffffffffu, incl <= want);        // (a prefix: sums ascend)
      const int skip = min(__popc(past), (units - 1) / 32);
      if (skip > 0) base_u = 32 * (skip - 1), items_here = __shfl_sync(0xffffffffu, incl, skip - 1);
    }
    uint32_t n = 0, st = 0, round = 0;                     // pairs so far, the next one's place, times around
    bool ok = true;
    for (;;) {
      int ticket = 0;
      if (!one && lane == 0) ticket = atomicAdd(p.w.ctr, 1);
      while (base_u + 32 < units && want >= items_before + items_here) {
        items_before += items_here, cuts_before += cuts_here, parts_before += parts_here;
        base_u += 32;
        mine = {0, 0, 0, 0, 0, 0};
        if (base_u + lane < units) mine = load_unit(p, base_u + lane);
        ranges = rows_cut >= mine.rows ? 1 : ceil_div(mine.rows, rows_cut);
        items = mine.pairs * ranges;
        const int cuts = ranges > 1 ? mine.pairs : 0, parts = cuts * ranges;
        items_pre = warp_incl_scan(items), cuts_pre = warp_incl_scan(cuts), parts_pre = warp_incl_scan(parts);
        items_here = __shfl_sync(0xffffffffu, items_pre, 31);
        cuts_here = __shfl_sync(0xffffffffu, cuts_pre, 31);
        parts_here = __shfl_sync(0xffffffffu, parts_pre, 31);
        items_pre -= items, cuts_pre -= cuts, parts_pre -= parts;
      }
      if (want >= items_before + items_here || (one && want >= slice_end)) break;
      const int here = want - items_before;
      const int src = __ffs((int)__ballot_sync(0xffffffffu, items_pre <= here && here < items_pre + items)) - 1;
      Unit u;
      u.cnt = __shfl_sync(0xffffffffu, mine.cnt, src), u.start = __shfl_sync(0xffffffffu, mine.start, src);
      u.len = __shfl_sync(0xffffffffu, mine.len, src), u.tok0 = __shfl_sync(0xffffffffu, mine.tok0, src);
      u.pairs = __shfl_sync(0xffffffffu, mine.pairs, src), u.rows = __shfl_sync(0xffffffffu, mine.rows, src);
      const int n_ranges = __shfl_sync(0xffffffffu, ranges, src);
      const int cut0 = cuts_before + __shfl_sync(0xffffffffu, cuts_pre, src);
      const int part0 = parts_before + __shfl_sync(0xffffffffu, parts_pre, src);
      const int rem = here - __shfl_sync(0xffffffffu, items_pre, src);
      const int range = one ? 0 : rem / u.pairs;
      const int p0 = one ? rem : rem - range * u.pairs, p1 = one ? min(u.pairs, rem + slice_end - want) : p0 + 1;
      const int range0 = n_ranges > 1 ? range * rows_cut : 0;
      const int range1 = n_ranges > 1 ? min(u.rows, range0 + rows_cut) : u.rows;
      const int unit = base_u + src;
      const int64_t list = (int64_t)unit * a.umax;
      const bool keep = one && u.len > u.tok0;
      const int last = u.len > 0 ? u.start + u.len - 1 : -1;
      // 32 entries at a time, those of the next time on their way
      const int two = 2 * chunks, per = 32 / two;          // pairs a time
      const int ents = min(u.cnt, p1 * two);
      RawEntry then = fetch_entry(a, list, p0 * two + lane, ents);
      for (int b = p0; ok && b < p1; b += per) {
        const Entry now = check_entry(a, then, b * two + lane < ents, last >> a.cs_log, staged);
        then = fetch_entry(a, list, (b + per) * two + lane, ents);
        for (int pr = b; pr < min(b + per, p1); ++pr, ++n) {
          const uint32_t rec = n % kRec;
          if (n >= kRec) ok = wait_warp(pair_free + 8 * rec, n / kRec - 1);
          if (round > 0) ok = ok && wait_warp(k_free + 8 * st, round - 1);
          if (!ok) break;
          Pair &r = x.pair[rec];
          const int from_lane = (pr - b) * two + (lane & (two - 1));
          const int slot = __shfl_sync(0xffffffffu, now.slot, from_lane), pos = __shfl_sync(0xffffffffu, now.pos, from_lane);
          if (lane < two) r.pos[lane] = pos, r.slot[lane] = slot;
          if (lane == 0) {
            r.unit = unit, r.start = u.start, r.len = u.len, r.last = last, r.tok0 = u.tok0;
            r.keep_q = keep ? (pr == p0 ? (pr == p1 - 1 ? 3 : 1) : (pr == p1 - 1 ? 2 : 4)) : 0;
            r.parts = n_ranges, r.part0 = part0 + pr * n_ranges, r.part = part0 + pr * n_ranges + range;
            r.cut = 2 * (cut0 + pr);
          }
          int r0 = 0;
          if (!keep) {
            // tokens before the pair's first row see none of it
            const int first = __reduce_min_sync(0xffffffffu, pos);
            r0 = min(max(range0, first == INT_MAX ? INT_MAX : max(0, first - u.start - u.tok0) / a.tt), range1);
          }
          if (lane == 0) r.r0 = r0, r.r1 = u.len > u.tok0 ? range1 : r0;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_expect_tx(pair_full + 8 * rec, 2 * kTileBytes);
            mbar_arrive(rec_full + 8 * rec);
          }
          __syncwarp();
          load_third(0, slot, pos, last, st, pair_full + 8 * rec);
          if (++st == kPair) st = 0, ++round;
        }
      }
      if (!ok) break;
      want = one ? want + p1 - p0 : __shfl_sync(0xffffffffu, ticket, 0) + cta;
    }
    if (ok) {
      const uint32_t rec = n % kRec;
      if (n >= kRec) ok = wait_warp(pair_free + 8 * rec, n / kRec - 1);
      if (ok && lane == 0) {
        x.pair[rec].unit = -1;
        mbar_arrive(rec_full + 8 * rec);
        mbar_arrive(pair_full + 8 * rec);
      }
    }
    // copies in flight are waited for before the CTA leaves (there are no more than those of the last kPair
    // pairs, whose records are not the last one's)
    for (uint32_t i = n >= kPair ? n - kPair : 0; i < n; ++i)
      mbar_wait(pair_full + 8 * (i % kRec), (i / kRec) & 1u, a.raised);
  } else if (warp == kSums + 2) {
    // ------------------------------------------------------ a third of a pair's keys
    uint32_t st = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const uint32_t rec = n % kRec;
      ok = wait_warp(rec_full + 8 * rec, n / kRec);
      if (!ok) break;
      const Pair &r = x.pair[rec];
      if (r.unit < 0) break;
      load_third(1, r.slot[lane & 15], r.pos[lane & 15], r.last, st, pair_full + 8 * rec);
      if (++st == kPair) st = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_free + 8 * rec);
    }
  } else if (warp == kSums + 3) {
    // ------------------------------------------- Q's tiles, and their log-sum-exps
    uint32_t nq = 0, st = 0;
    bool ok = true;
    // a lane's four rows of a tile: their tokens (-1: none) and places
    int mine[4], off[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = lane + 32 * k, tok = e / a.G;
      mine[k] = e < rows_tile ? tok : -1;
      off[k] = tok * a.Hq + e - tok * a.G;
    }
    for (uint32_t n = 0; ok; ++n) {
      const uint32_t rec = n % kRec;
      ok = wait_warp(rec_full + 8 * rec, n / kRec);
      if (!ok) break;
      const Pair &r = x.pair[rec];
      const int unit = r.unit;
      if (unit < 0) break;
      load_third(2, r.slot[lane & 15], r.pos[lane & 15], r.last, st, pair_full + 8 * rec);
      if (++st == kPair) st = 0;
      const int r1 = r.r1, tok0 = r.tok0, len = r.len, b = unit / a.Hkv, h0 = unit % a.Hkv * a.G;
      if (new_q(r.keep_q)) {
        // (log-sum-exps are loaded two tiles ahead)
        const float *from = p.lse + ((int64_t)b * a.T + tok0) * a.Hq + h0;
        auto fetch = [&](int t, float (&v)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = -INFINITY;
            if (t < r1 && mine[k] >= 0 && tok0 + t * a.tt + mine[k] < len) v[k] = from[(int64_t)t * a.tt * a.Hq + off[k]];
          }
        };
        float v[2][4];
        fetch(r.r0, v[0]), fetch(r.r0 + 1, v[1]);
        for (int t = r.r0; t < r1; ++t, ++nq) {
          const uint32_t sq = nq % kQ;
          if (nq >= kQ) ok = wait_warp(q_free + 8 * sq, nq / kQ - 1);
          if (!ok) break;
          // a row without keys (-inf) has no weights, nor has what is no row: 2^-inf
#pragma unroll
          for (int k = 0; k < 4; ++k) x.lse[sq][lane + 32 * k] = v[0][k] == -INFINITY ? -INFINITY : v[0][k] * -1.4426950408889634f;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(q_full + 8 * sq, (uint32_t)(rows_tile * 256));
          __syncwarp();
          if (lane < 2)
            tma_load_4d(q0 + (sq * 2 + lane) * q_half, &p.q, 64 * lane, h0, tok0 + t * a.tt, b, q_full + 8 * sq);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[0][k] = v[1][k];
          fetch(t + 2, v[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_free + 8 * rec);
    }
    for (uint32_t i = nq >= kQ ? nq - kQ : 0; i < nq; ++i) mbar_wait(q_full + 8 * (i % kQ), (i / kQ) & 1u, a.raised);
  } else if (warp == kSums) {
    // -------------------------------------------------------------------- products
    const uint32_t id = idesc_bf16(128, (rows_tile + 31) / 32 * 32, 0, 0);   // (as many columns as are read)
    const uint64_t q_desc = smem_desc_sw128(q0, 16, 1024), k_desc = smem_desc_sw128(k0, 16, 1024);
    uint32_t nq = 0, ns = 0, st = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const uint32_t rec = n % kRec;
      ok = wait_warp(pair_full + 8 * rec, n / kRec);
      if (!ok) break;
      const Pair &r = x.pair[rec];
      if (r.unit < 0) break;
      const int r1 = r.r1, keep = r.keep_q;
      for (int t = r.r0; t < r1; ++t, ++ns) {
        if (new_q(keep)) ok = wait_warp(q_full + 8 * (nq % kQ), nq / kQ);
        if (!ok) break;
        const uint32_t sq = nq % kQ, buf = ns & 1u;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (ns >= 2) ok = wait_warp(s_free + 8 * (2 * w + buf), (ns >> 1) - 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_lane()) {
            const uint64_t qb = q_desc + sq * (q_half / 8), kb = k_desc + (st * 2 + w) * (kTileBytes / 16);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              tc_mma(tmem + 256 * w + 128 * buf, kb + ((ks >> 2) * kTileHalfBytes + (ks & 3) * 32) / 16,
                     qb + ((ks >> 2) * q_half + (ks & 3) * 32) / 16, id, ks > 0);
            }
            mbar_arrive(s_full + 8 * (2 * w + buf));       // (hands on the pair's and the queries' records)
            tc_commit(s_full + 8 * (2 * w + buf));
            if (w == 1 && last_q(keep)) tc_commit(q_free + 8 * sq);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (last_q(keep)) ++nq;
      }
      if (!ok) break;
      if (elect_lane()) tc_commit(k_free + 8 * st);
      if (++st == kPair) st = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_free + 8 * rec);
    }
    if (elect_lane()) tc_commit(mma_done);
    __syncwarp();
    mbar_wait(mma_done, 0, a.raised);
  } else {
    // ------------------------------------------------------- exponentials and sums
    const int w = warp >> 2, quarter = warp & 3, key = 32 * quarter + lane;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const int key_chunk = w * chunks + (key >> a.cs_log), key_row = key & (a.cs - 1);
    // the chunk's first key writes its weight
    const bool writes = key_row == 0;
    uint32_t nq = 0, ns = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const uint32_t rec = n % kRec;
      ok = wait_warp(pair_full + 8 * rec, n / kRec);
      if (!ok) break;
      const Pair &r = x.pair[rec];
      const int unit = r.unit;
      if (unit < 0) break;
      const int r0 = r.r0, r1 = r.r1, keep = r.keep_q, first = r.pos[key_chunk];
      // the key's place among the counted tokens (those at or behind it see it), and how many there are
      const int place = first == INT_MAX ? INT_MAX : first + key_row - r.start - r.tok0, counted = r.len - r.tok0;
      // what the chunk holds so far is on its way meanwhile
      float *const to = p.weight + (int64_t)unit * a.C + (first == INT_MAX ? 0 : first >> a.cs_log);
      const int parts = r.parts;
      const float old = writes && first != INT_MAX && p.decay != 0.f && parts == 1 ? *to : 0.f;
      float total = 0.f;
      for (int t = r0; t < r1; ++t, ++ns) {
        const uint32_t sq = nq % kQ, buf = ns & 1u;
        ok = wait_warp(s_full + 8 * (2 * w + buf), ns >> 1);
        if (!ok) break;
        tc_fence_after();
        const int tok = t * a.tt;                          // of the tile's first row
        const int cols = min(rows_tile, (counted - tok) * a.G);
        // columns of tokens that see the key; S of the others may be anything
        const int lo = place <= tok ? 0 : (place - tok >= a.tt ? 128 : (place - tok) * a.G);
        // every column that is read counts.  (Columns behind the tile's last query row do not: they are 0 times the key,
        // NaN where the key is infinite.)
        const bool whole = __all_sync(0xffffffffu, lo == 0 && cols == rows_tile && (cols & 31) == 0);
        const float *ls = x.lse[sq];
        const uint32_t at = tmem + lane_base + 256 * w + 128 * buf;
        // 32 columns at a time, the next ones on their way
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        float s[2][32], y[32];
        tmem_ld32(at, s[0]);
        // (two loops: with the choice by blocks inside one, 2,048 tokens of 64 heads took 1,156 us, so 1,024)
        auto fetched = [&](int h) {
          tmem_wait_ld();
          tmem_ready(s[h & 1]);
          if (h < 3 && 32 * h + 32 < cols) tmem_ld32(at + 32 * h + 32, s[(h + 1) & 1]);
        };
        // the weights of columns 32 h + 4 e and three more
        auto four = [&](int h, int e) {
          const float *v = s[h & 1];
          const float4 z = *reinterpret_cast<const float4 *>(ls + 32 * h + 4 * e);
          const float2 y0 = fma2(make_float2(v[4 * e], v[4 * e + 1]), make_float2(a.sl2, a.sl2), make_float2(z.x, z.y));
          const float2 y1 = fma2(make_float2(v[4 * e + 2], v[4 * e + 3]), make_float2(a.sl2, a.sl2), make_float2(z.z, z.w));
          y[4 * e] = ex2_approx(y0.x), y[4 * e + 1] = ex2_approx(y0.y);
          y[4 * e + 2] = ex2_approx(y1.x), y[4 * e + 3] = ex2_approx(y1.y);
        };
        if (whole) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            if (32 * h >= cols) break;
            fetched(h);
#pragma unroll
            for (int e = 0; e < 8; ++e) four(h, e);
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[e & 1] = add2(sum[e & 1], make_float2(y[2 * e], y[2 * e + 1]));
          }
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            if (32 * h >= cols) break;
            fetched(h);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (32 * h + 4 * e >= cols) break;
              four(h, e);
#pragma unroll
              for (int k = 4 * e; k < 4 * e + 4; ++k) y[k] = 32 * h + k >= lo && 32 * h + k < cols ? y[k] : 0.f;
              sum[0] = add2(sum[0], make_float2(y[4 * e], y[4 * e + 1]));
              sum[1] = add2(sum[1], make_float2(y[4 * e + 2], y[4 * e + 3]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(s_free + 8 * (2 * w + buf));
          if (last_q(keep)) mbar_arrive(q_free + 8 * sq);
        }
        if (last_q(keep)) ++nq;
        total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      // a chunk's rows, across lanes; those of 64 in two warps
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (a.cs > 16) total += __shfl_xor_sync(0xffffffffu, total, 16);
      if (a.cs > 32) {
        if (lane == 0) x.sum[n & 1u][w][quarter] = total;
        // (a wait that gives up: a warp may have done so already, before an event that the others still saw)
        __syncwarp();
        if (lane == 0) mbar_arrive(summed + 8 * w);
        ok = wait_warp(summed + 8 * w, n);
        if (!ok) break;
        total = x.sum[n & 1u][w][quarter & 2] + x.sum[n & 1u][w][quarter | 1];
      }
      if (parts == 1) {
        if (writes && first != INT_MAX) *to = p.decay == 0.f ? total : fmaf(p.decay, old, total);
      } else {
        const int part0 = r.part0, part = r.part, cut = r.cut;
        if (writes) __stcg(p.parts + (int64_t)part * 16 + w * 8 + (key >> a.cs_log), total);
        __syncwarp();
        int last = 0;
        if (lane == 0) {
          __threadfence();
          int32_t *ctr = p.w.ctr + 2 + cut + w;
          last = atomicAdd(ctr, 1) == 4 * parts - 1;       // (four warps a part)
          if (last) *ctr = 0;
          __threadfence();
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        __syncwarp();
        const int at = last && lane < chunks ? r.pos[w * chunks + lane] : INT_MAX;
        if (at != INT_MAX) {
          float v = 0.f;
          for (int i = 0; i < parts; ++i) v += __ldcg(p.parts + (int64_t)(part0 + i) * 16 + w * 8 + lane);
          float *const all = p.weight + (int64_t)unit * a.C + (at >> a.cs_log);
          *all = p.decay == 0.f ? v : fmaf(p.decay, *all, v);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_free + 8 * rec);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSums) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
  }
  leave_counters(p.w, a, &x.pending);
}

}  // namespace

int64_t weights_workspace(int sm_count) {
  return (int64_t)2 * kItemsPerCta * sm_count * 16 * 4;
}

cudaError_t launch_weights(const WeightsArgs &e, cudaStream_t stream) {
  const PagesArgs &a = e.p;
  WeightsParams p{};
  p.a = a;
  const int most = 128 / a.G, seen = e.window > 0 && e.window < a.T ? e.window : a.T;
  p.a.tt = seen < 1 ? 1 : (seen < most ? seen : most);
  const bool hot = a.hot_slots > 0, far = a.max_misses > 0;
  // (without tokens nothing is read through the map)
  const int64_t dense[3] = {(int64_t)a.Hq * kD, (int64_t)a.Hq * kD, kD};
  if (!make_rows_map(&p.q, a.T > 0 ? e.q : e.dummy, a.T > 0 ? e.q_stride : dense, a.B, a.T > 0 ? a.T : 1, a.Hq, a.G, p.a.tt) ||
      !make_pages_map(&p.k, hot ? e.Khot : e.dummy, hot ? a.hot_slots : 1, a.cs) ||
      !make_pages_map(&p.kst, far ? e.Kst : e.dummy, far ? a.max_misses : 1, a.cs))
    return cudaErrorInvalidValue;
  p.lse = e.lse, p.weight = e.weight, p.window = e.window, p.decay = e.decay, p.parts = e.parts;
  p.w = {e.ctr, kCtrPerCta * e.sm_count};
  cudaError_t r = set_dyn_smem((const void *)k_weights, kSmem);
  if (r != cudaSuccess) return r;
  return launch_k(k_weights, dim3(e.sm_count), dim3(kThreads), kSmem, stream, p);
}

}  // namespace dd
