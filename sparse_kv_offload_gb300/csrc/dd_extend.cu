// Attention of new tokens over a paged cache, on the fifth-generation tensor cores.
//
// Token t of request b stands at position p = start[b] + t and sees the rows of its KV
// head's listed chunks whose positions are at most p:  o = sum_i w_i v_i / sum_i w_i with
// w_i = exp(scale q.k_i), and lse = ln sum_i w_i.  One pass over the rows: with a reference m of
// the scores seen so far, l = sum exp(s - m) and O = sum exp(s - m) v are kept, and both are
// multiplied by exp(m - m') where m moves (only when a score exceeds it by 2^8: the weights
// then stay finite, and few tiles pay).
//
// The G heads of a KV head share its rows, so a tile of 128 query rows is tt = 128 / G tokens
// by G heads, brought by TMA from the caller's strides.  A CTA (one per SM) works on two
// streams, each with S (128 x 128) and O (128 x 128) in tensor memory and four softmax warps,
// a thread a query row; while one stream's softmax runs, the other's products do.  With
// more than 128 query rows per KV head the streams are two row tiles over the same keys; with
// fewer they are the even and the odd tiles of keys of one row tile, joined at the end.
//   warps 0-3, 4-7  softmax of the streams: S out of tensor memory, weights back in
//                   its place, O rescaled when a reference moves, outputs
//   warp 8          S = Q K^T, O += P V (P straight from tensor memory)
//   warp 9          hands out the work and brings K's tiles, warp 10 Q's and V's
//   warp 11         looks over V's tiles that some row does not see entirely: a masked weight of
//                   0 times an infinity or NaN would be NaN, so such values are taken out of the
//                   tile, and a row that does see one has it put into its output at the end
// Weights are rounded to bf16 for the second product (V's type: the tensor cores take two
// operands of one type): up to 2^-8 of each weight, at random, as the rounding of the
// output.  With up to 32 query rows (kLowRows), where one warp of a stream's four has rows, what the rounding
// leaves out is a second operand in the other half of S's columns: 2^-15 of each weight, much as the attentions
// over a step's selection have it.  With it and without: 16 whole caches 222 and 216 us, outputs off by 0.0016 and
// 0.0023 (relative L2; 0.0016 is their own rounding); 40 query rows 69 and 61; prompts 436 and 305; 2,048
// tokens behind 62K 4.2 and 2.8 ms.  l is the sum of the weights before that, so that lse has fp32's precision.
//
// Work: with two row tiles an item is a pair of them, whole or by a range of tiles of keys (cut_of); items are
// handed out one after another, the pairs of one KV head and range next to each other, so that the CTAs
// at work read the same keys at about the same time, out of L2.  With one row tile a unit a CTA has
// an equal slice of all units' tiles, as nothing is read twice and the bytes bound it (decode 256 us, 435 with
// ranges).  A row tile that is cut has its parts joined by whoever finishes last, in the ranges' order.
//
// What bounds it: HBM with one token a request (16 whole caches of up to 32K: 216 to 245 us by their lengths, 6,500
// GB/s); with many, the tensor cores and beside them the issue slots of the softmax (2,048 tokens behind 62K
// others, 64 heads: 2.81 ms, 1,540 TFLOP/s; a step of two tiles takes 3,000 cycles, its products 2,500 at the rate
// of a large product).  Short items pay for their ends, some 12,000 cycles each: the last weights, O out of tensor
// memory, places and stores (first 2,048 tokens of four prompts, 64 heads: 304 us, 906 TFLOP/s).  The softmax's loop needs nearly all of its registers:
// anything that the compiler keeps across it, an item's end that holds 64 columns at once among it, costs 20 to 60%.
#include "dd_pages.cuh"

namespace dd {

namespace {

constexpr int kThreads = 384;
constexpr int kK = 3;                                // tiles of K on the way
constexpr int kInfo = 8;                             // records of K's tiles (a softmax warp is at most kK + 2 behind)
constexpr uint32_t kTmem = 512;                      // S: 2 x 128 columns, O: 2 x 128
constexpr int kSoftRegs = 208, kOtherRegs = 80;      // 256 * 208 + 128 * 80 <= 384 * 168 at launch
constexpr float kHead = 8.f;                         // weights stay below 2^8
constexpr int kLowRows = 32;                         // query rows of a tile whose weights have two parts

struct Item {
  int unit, b, h0, t0, start, len;   // the unit's request and first query head
  int j0;                     // first tile of keys
  int ents;                   // the list's entries that the item's last token may see
  int pos_max, pos_min;       // positions of the item's last and first token
  int c[2];                   // tiles of each stream
  int parts[2];               // of each stream's row tile: 0 nothing to write, 1 its outputs, more: a part to be joined
  int64_t part0, part;        // slots of the first range's parts and of this one's (slices: the first slice's number)
  int cut;                    // arrival counter (pairs: and the next one)
};

// A row tile to be joined.
struct Task {
  int unit, len, token, parts;    // its first token
  int64_t first;
};
constexpr int kTasks = 16;    // of a CTA: with fewer than four left its next item is its last (eight cut items a CTA; there are five)

struct Misc {
  uint64_t bars[40];
  Item item[2];
  int pos[kInfo][8];          // positions of the first rows of a tile's chunks
  int whole[kInfo];           // every query row sees the whole tile
  int vpos[3][8], vwhole[3];  // the same of V's tiles
  int bad[3][128];            // lowest position of a NaN, +inf, -inf in each column of V
  Task task[kTasks];
  uint32_t sum[kThreads / 32], block[32];   // units' groups, or tiles and costs: of each warp, of the first blocks of 32
  int tasks, bad_item, dead, pending;
  uint32_t tmem;
};

constexpr size_t kTiles = (size_t)(2 + kK + 2) * kTileBytes;   // queries of two row tiles, or of one and a third tile of V
constexpr size_t kSmem = kTiles + sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory of a CTA");

struct ExtendParams {
  CUtensorMap q, k, v, kst, vst;
  PagesArgs a;
  uint16_t *out;
  int64_t os[3];
  float *lse;
  float *part_o;              // [slots][rows][128]
  float2 *part_ml;            // [slots][rows]: reference (a score before the factor), sum
  WorkCounters w;
  bool wide;                  // rows of `out` begin at multiples of 32 bytes
  int mt;                     // tokens of an item
};

// One (request, KV head) as the planning sees it.
struct Unit {
  int cnt, start, len, groups, tiles;     // groups of mt tokens; tiles of keys that the last of them may see
};

// entries that a token may see: chunk numbers ascend, so entry i is chunk i or a later one
__device__ __forceinline__ int entry_bound(const PagesArgs &a, const Unit &u, int token) {
  return min(u.cnt, ((u.start + token) >> a.cs_log) + 1);
}

__device__ __forceinline__ int tiles_of(const PagesArgs &a, int entries) {
  return max(1, ((entries << a.cs_log) + kTileKeys - 1) / kTileKeys);      // (a row without keys still has its zeros to write)
}

__device__ __forceinline__ Unit load_unit(const ExtendParams &p, int u) {
  Unit r = {0, 0, 0, 0, 0};
  const Request q = load_request(p.a, u / p.a.Hkv);
  r.cnt = load_count(p.a, u);
  r.start = q.start, r.len = q.len;
  r.groups = ceil_div(q.len, p.mt);
  if (r.groups) r.tiles = tiles_of(p.a, entry_bound(p.a, r, q.len - 1));
  return r;
}

// The first group of tokens that has more than `tiles` tiles of keys.
__device__ __forceinline__ int first_longer(const ExtendParams &p, const Unit &u, int tiles) {
  if (tiles <= 0) return 0;
  if (u.tiles <= tiles) return u.groups;
  const int need = tiles * kTileKeys - u.start + 1;        // its last token's number, from 1
  return need <= 0 ? 0 : ceil_div(need, p.mt) - 1;
}

// A unit without its last `whole` groups of tokens.
__device__ __forceinline__ Unit cut_part(const ExtendParams &p, const Unit &u, int whole) {
  Unit r = u;
  r.groups -= whole;
  r.tiles = r.groups ? tiles_of(p.a, entry_bound(p.a, u, min(r.groups * p.mt, u.len) - 1)) : 0;
  return r;
}

// Pairs of row tiles: as many as there are whole rounds of CTAs for are taken whole, in order, and the
// rest, fewer than CTAs, is cut into ranges of at most this many tiles of keys: of 1/s of the longest pair
// for s = 1, 2, .. the one that ends first, by rounds of items, each its tiles and kItemCost of them for what an
// item costs beside (queries, sums out and in), and kJoinCost for the joins at the end.  With P CTAs: pairs that are cut < P, their ranges
// <= work / length + pairs <= 5 P.
constexpr int kItemCost = 3, kJoinCost = 12, kItemsPerCta = 4;
__device__ __forceinline__ int cut_of(int work, int groups, int longest, int cta, int lane) {
  if (groups == 0) return 1;
  const int least = max(1, ceil_div(work, kItemsPerCta * cta));
  // (fewer groups than CTAs and at most 8,192 tiles each: costs stay below 2^17, lengths below 2^14)
  uint32_t best = ~0u;
  for (int s = 1 + lane; s <= longest; s += 32) {
    const int len = max(ceil_div(longest, s), least);
    const int items = min(groups * ceil_div(longest, len), (int)((unsigned)work / (unsigned)len) + groups);
    const int cost = ceil_div(items, cta) * (len + kItemCost) + (len < longest ? kJoinCost : 0);
    best = min(best, (uint32_t)cost << 14 | (uint32_t)(16383 - len));
    if (len == least) break;
  }
  return 16383 - (int)(__reduce_min_sync(0xffffffffu, best) & 16383u);
}

// One row tile a unit: the units' tiles of keys, laid end to end, are cut into equal slices, one a CTA; kUnitCost
// tiles stand before each unit's for what it costs beside.  A unit that slices cut is joined from a part of
// each: in its first slice it is the last unit, in the others the first.
constexpr int kUnitCost = 2;

// A row tile that has several parts: o = sum_q f_q O_q / sum_q f_q l_q with f_q = 2^((m_q - m) sl2), m the largest
// reference, in the order of the parts.
struct Join {
  const float *part_o;
  const float2 *part_ml;
  int64_t first;
  int pairs, parts, rows, rows_tile, G, Hq;
  float scale, sl2;
  uint16_t *out;              // the row tile's first row
  int64_t os1, os2;
  float *lse;
};

__device__ __forceinline__ int64_t slice_slot(int64_t slice, bool first) { return 2 * slice + (first ? 1 : 0); }

// R rows by Q parts are on their way at once, the next rows' while these are written; lane (32 / R) j + q
// holds the statistics of row j's part q.
template <int R, int Q>
__device__ __forceinline__ void join_rows(const Join &p, int join_w, int join_n) {
  constexpr int L = 32 / R;
  const int lane = threadIdx.x & 31, lj = lane / L, lq = lane % L;
  const int rows = p.rows, n_parts = p.parts;
  auto slot_of = [&](int q) -> int64_t {
    return p.pairs == 2 ? p.first + 2 * q : slice_slot(p.first + q, q == 0);
  };
  auto stats = [&](int k, int q) {
    return q < n_parts ? __ldcg(p.part_ml + slot_of(q) * p.rows_tile + k) : make_float2(-INFINITY, 0.f);
  };
  float4 v[R][Q];
  float2 ml;
  auto load = [&](int k0, int q0) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float *from = p.part_o + slot_of(min(q0 + q, n_parts - 1)) * p.rows_tile * kD + 4 * lane;
#pragma unroll
      for (int j = 0; j < R; ++j) v[j][q] = __ldcg(reinterpret_cast<const float4 *>(from + min(k0 + j, rows - 1) * kD));
    }
  };
  int k0 = R * join_w;
  if (k0 < rows) load(k0, 0), ml = stats(min(k0 + lj, rows - 1), lq);
  while (k0 < rows) {
    const int k = min(k0 + lj, rows - 1);
    float top = ml.x;
    for (int q = lq + L; q < n_parts; q += L) top = fmaxf(top, stats(k, q).x);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f, f = 0.f;
    float4 acc[R];
#pragma unroll
    for (int j = 0; j < R; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q0 = 0; q0 < n_parts; q0 += Q) {
      if (q0 > 0) load(k0, q0);
      if (q0 % L == 0) {
        if (q0 > 0) ml = stats(k, q0 + lq);
        f = ex2_approx((ml.x - ref) * p.sl2);
        total += f * ml.y;
      }
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const float fq = __shfl_sync(0xffffffffu, f, L * j + q0 % L + q);
          if (q0 + q < n_parts) {
            acc[j].x += fq * v[j][q].x, acc[j].y += fq * v[j][q].y;
            acc[j].z += fq * v[j][q].z, acc[j].w += fq * v[j][q].w;
          }
        }
    }
    const int kn = k0 + R * join_n;
    if (kn < rows) load(kn, 0), ml = stats(min(kn + lj, rows - 1), lq);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int t = k / p.G, h = k - t * p.G;
    const int64_t to = t * p.os1 + h * p.os2;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float iv = __shfl_sync(0xffffffffu, inv, L * j);
      const int64_t at = __shfl_sync(0xffffffffu, to, L * j);
      if (k0 + j < rows)
        *reinterpret_cast<uint2 *>(p.out + at + 4 * lane) =
            make_uint2(cvt_bf16x2(acc[j].x * iv, acc[j].y * iv), cvt_bf16x2(acc[j].z * iv, acc[j].w * iv));
    }
    if (p.lse && lq == 0 && k0 + lj < rows)
      p.lse[(int64_t)t * p.Hq + h] = total == 0.f ? -INFINITY : (top == -INFINITY ? NAN : top * p.scale + logf(total));
    k0 = kn;
  }
}

// kPairs: row tiles of an item.  kLow: the weights' second parts.
template <int kPairs, bool kLow>
__global__ void __launch_bounds__(kThreads, 1) k_extend(const __grid_constant__ ExtendParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc &x = *reinterpret_cast<Misc *>(smem + kTiles);
  const PagesArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // tiles of V on the way: with few rows a tile is held longest (its scores and weights come first), and the second
  // row tile's place is free (16 whole caches: 222 us with three, 226 with two)
  constexpr int kV = kLow ? 3 : 2;
  const uint32_t q0 = smem_u32(smem), k0 = q0 + (kLow ? 1 + kV : 2) * kTileBytes;
  const uint32_t v0 = kLow ? q0 + kTileBytes : k0 + kK * kTileBytes;
  const uint32_t bars = smem_u32(x.bars);
  const uint32_t k_full = bars, k_free = k_full + 8 * kK, v_full = k_free + 8 * kK, v_ok = v_full + 8 * kV,
                 v_free = v_ok + 8 * kV, q_full = v_free + 8 * kV, q_free = q_full + 8, s_full = q_free + 8,
                 p_half = s_full + 16, p_ready = p_half + 16, o_full = p_ready + 16, item_full = o_full + 16, item_free = item_full + 16,
                 looked = item_free + 16, handed = looked + 16, taken = handed + 8, mma_done = taken + 8, stored = mma_done + 8;
  if (tid == 0) {
    for (int i = 0; i < kK; ++i) mbar_init(k_full + 8 * i, 1), mbar_init(k_free + 8 * i, 1);
    for (int i = 0; i < kV; ++i) mbar_init(v_full + 8 * i, 1), mbar_init(v_ok + 8 * i, 1), mbar_init(v_free + 8 * i, 1);
    mbar_init(q_full, 1), mbar_init(q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(looked + 8 * i, 1), mbar_init(s_full + 8 * i, 2), mbar_init(p_half + 8 * i, 4), mbar_init(p_ready + 8 * i, 4), mbar_init(o_full + 8 * i, 1);
      mbar_init(item_full + 8 * i, 1), mbar_init(item_free + 8 * i, 11), mbar_init(stored + 8 * i, 4);
    }
    mbar_init(handed, 4), mbar_init(taken, 4), mbar_init(mma_done, 1);
    x.bad_item = -1, x.dead = 0, x.tasks = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&x.tmem)), "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  pdl_wait();
  pdl_trigger();
  if (tid == 0) x.pending = load_status(a.status);
  // groups of all units, or their tiles and costs (below 2^31): a warp's blocks of 32 units each
  const int units = a.B * a.Hkv;
  constexpr bool sliced = kPairs == 1;
  Unit few = {0, 0, 0, 0, 0};                              // a lane's unit, where there are no more than 32
  if (units <= 32 && lane < units && (warp == 0 || warp == 9)) few = load_unit(p, lane);
  {
    uint32_t total = 0;
    for (int u0 = 32 * warp; u0 < units; u0 += kThreads) {
      const Unit r = units <= 32 ? few : (u0 + lane < units ? load_unit(p, u0 + lane) : Unit{0, 0, 0, 0, 0});
      const uint32_t sum = __reduce_add_sync(0xffffffffu, (uint32_t)(sliced ? (r.groups ? r.tiles + kUnitCost : 0) : r.groups));
      if (lane == 0 && u0 < 1024) x.block[u0 >> 5] = sum;
      total += sum;
    }
    if (lane == 0) x.sum[warp] = total;
  }
  __syncthreads();
  tc_fence_after();
  const bool pending = x.pending != 0;      // an error is pending: no work
  const uint32_t tmem = x.tmem;
  const int rows_tile = a.tt * a.G;         // query rows of a tile
  const int chunks = kTileKeys / a.cs;      // of a tile

  auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_or_dead(bar, parity, &x.dead, a.raised));
  };

  // (with an error pending: nothing, but the counters below are left all the same)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (pending) {
    } else if (warp == 9) {
      // ------------------------------------------------------- the work, and K's tiles
      const int cta = (int)gridDim.x;
      uint32_t total = lane < kThreads / 32 ? x.sum[lane] : 0u;
      total = __reduce_add_sync(0xffffffffu, total);
      const int whole_groups = (int)(total / cta * cta);
      int cut = 1;
      if (!sliced) {
        // what is left to cut
        int work = 0, longest = 0, before = 0;
        for (int u0 = 0; u0 < units; u0 += 32) {
          Unit r = {0, 0, 0, 0, 0};
          if (u0 + lane < units) r = units <= 32 ? few : load_unit(p, u0 + lane);
          const int incl = warp_incl_scan(r.groups);
          r = cut_part(p, r, min(r.groups, max(0, whole_groups - before - (incl - r.groups))));
          work += r.groups * r.tiles;
          longest = max(longest, r.tiles);
          before += __shfl_sync(0xffffffffu, incl, 31);
        }
        work = __reduce_add_sync(0xffffffffu, work);
        longest = __reduce_max_sync(0xffffffffu, longest);
        cut = cut_of(work, (int)total - whole_groups, longest, cta, lane);
      }
      const int per = max((int)((total + cta - 1) / cta), 2);      // of a slice: a tile for each stream at least
      const int64_t staged = staged_slots(a);

      // The lanes hold 32 units; counts before them and of them.  Slices: `items` are tiles (and costs), the place that
      // is wanted moves through the CTA's own slice.  Else items are handed out by tickets, the first by number.
      int base_u = -32, cuts_before = 0, parts_before = 0, parts_here = 0, cuts_here = 0;
      int items_before = 0, items_here = 0, groups_before = 0, groups_here = 0;
      Unit mine = {0, 0, 0, 0, 0}, rest = {0, 0, 0, 0, 0};  // a unit, and its groups that are cut
      int ranges = 0, items = 0, items_pre = 0, parts_pre = 0, cuts_pre = 0, m1 = 0;
      int want = sliced ? (int)blockIdx.x * per : (int)blockIdx.x;
      const int slice_end = want + per;
      if (sliced && units <= 1024) {
        // the block of units that the slice begins in
        const int incl = warp_incl_scan(32 * lane < units ? (int)x.block[lane] : 0);
        const uint32_t past = __ballot_sync(0xffffffffu, incl <= want);      // (a prefix: sums ascend)
        const int skip = min(__popc(past), (units - 1) / 32);
        if (skip > 0) base_u = 32 * (skip - 1), items_here = __shfl_sync(0xffffffffu, incl, skip - 1);
      }
      uint32_t n_item = 0, kt = 0;
      int tasks = 0;                                       // that this CTA may have to do
      bool ok = true;
      while (ok) {
        int ticket = INT_MAX / 2;
        // the next one: on its way during this one's work
        if (!sliced && lane == 0 && tasks + 4 <= kTasks) ticket = atomicAdd(p.w.ctr, 1);
        while (base_u + 32 < units && want >= items_before + items_here) {
          items_before += items_here, parts_before += parts_here, cuts_before += cuts_here, groups_before += groups_here;
          base_u += 32;
          mine = {0, 0, 0, 0, 0};
          if (base_u + lane < units) mine = units <= 32 ? few : load_unit(p, base_u + lane);
          int parts = 0, cuts = 0;
          if (sliced) {
            items = mine.groups ? mine.tiles + kUnitCost : 0;
          } else {
            const int groups_incl = warp_incl_scan(mine.groups);
            groups_here = __shfl_sync(0xffffffffu, groups_incl, 31);
            const int whole = min(mine.groups, max(0, whole_groups - groups_before - (groups_incl - mine.groups)));
            rest = cut_part(p, mine, whole);
            ranges = rest.groups ? ceil_div(rest.tiles, cut) : 0;
            m1 = first_longer(p, rest, cut);
            items = whole + rest.groups * min(ranges, 1);
            for (int s = 1; s < ranges; ++s) items += rest.groups - first_longer(p, rest, s * cut);
            parts = ranges > 1 ? items - whole - m1 : 0, cuts = ranges > 1 ? rest.groups - m1 : 0;
          }
          items_pre = warp_incl_scan(items), parts_pre = warp_incl_scan(parts), cuts_pre = warp_incl_scan(cuts);
          items_here = __shfl_sync(0xffffffffu, items_pre, 31);
          parts_here = __shfl_sync(0xffffffffu, parts_pre, 31);
          cuts_here = __shfl_sync(0xffffffffu, cuts_pre, 31);
          items_pre -= items, parts_pre -= parts, cuts_pre -= cuts;
        }
        const bool end = want >= items_before + items_here || (sliced && want >= slice_end);
        int src = 0, here = 0;
        if (!end) {
          // the unit that has it
          here = want - items_before;
          src = __ffs((int)__ballot_sync(0xffffffffu, items_pre <= here && here < items_pre + items)) - 1;
          here -= __shfl_sync(0xffffffffu, items_pre, src);
        }
        Unit u;
        u.cnt = __shfl_sync(0xffffffffu, mine.cnt, src), u.start = __shfl_sync(0xffffffffu, mine.start, src);
        u.len = __shfl_sync(0xffffffffu, mine.len, src), u.groups = __shfl_sync(0xffffffffu, mine.groups, src);
        u.tiles = __shfl_sync(0xffffffffu, mine.tiles, src);
        int m = 0, tiles = 0, j0 = 0, j1 = 0, n_cut = 1;    // group, its tiles, the range, how many ranges
        int64_t part0 = 0, part = 0;                        // slots of the pair's first part and of the range's
        int cut_no = 0;
        if (!end && sliced) {
          const int first = want - here;                    // where the unit begins
          const int upto = min(slice_end, first + kUnitCost + u.tiles);
          tiles = u.tiles;
          j0 = max(0, here - kUnitCost), j1 = max(0, upto - first - kUnitCost);
          const int s0 = (first + kUnitCost) / per, s1 = (first + kUnitCost + u.tiles - 1) / per;
          n_cut = s1 - s0 + 1, cut_no = s0;
          part0 = s0, part = slice_slot(blockIdx.x, (int)blockIdx.x == s0);
          want = upto;
          if (j0 >= j1) continue;                           // only of the cost before its tiles
        } else if (!end) {
          Unit r;
          r.cnt = u.cnt, r.start = u.start, r.len = u.len;
          r.groups = __shfl_sync(0xffffffffu, rest.groups, src), r.tiles = __shfl_sync(0xffffffffu, rest.tiles, src);
          const int n_ranges = __shfl_sync(0xffffffffu, ranges, src), um1 = __shfl_sync(0xffffffffu, m1, src);
          const int part_base = parts_before + __shfl_sync(0xffffffffu, parts_pre, src);
          const int cut_base = cuts_before + __shfl_sync(0xffffffffu, cuts_pre, src);
          const int whole = u.groups - r.groups;
          int s = 0;
          if (here < whole) {
            m = u.groups - 1 - here;                        // long ones first
          } else {
            int rem = here - whole;
            for (;; ++s) {
              const int n = r.groups - first_longer(p, r, s * cut);
              if (rem < n) break;
              rem -= n;
            }
            m = r.groups - 1 - rem;
          }
          tiles = tiles_of(a, entry_bound(a, u, min((m + 1) * p.mt, u.len) - 1));
          if (here < whole) {
            j1 = tiles;
          } else {
            n_cut = ceil_div(tiles, cut);
            j0 = s * cut, j1 = min(tiles, j0 + cut);
            int skip = 0;                                   // ranges of the groups before this one
            if (n_cut > 1)
              for (int k = 0; k < n_ranges; ++k) skip += max(0, m - max(first_longer(p, r, k * cut), um1));
            part0 = 2 * (part_base + skip), part = part0 + 2 * s;
            cut_no = 2 * (cut_base + m - um1);
          }
        }
        const uint32_t slot = n_item & 1u;
        if (n_item >= 2) ok = wait_warp(item_free + 8 * slot, (n_item >> 1) - 1);
        if (!ok) break;
        Item &it = x.item[slot];
        if (end) {
          if (lane == 0) {
            it.unit = -1;
            mbar_arrive(item_full + 8 * slot);
          }
          break;
        }
        const int unit = base_u + src;
        const int64_t list = (int64_t)unit * a.umax;
        const int t0 = m * p.mt, t_end = min(t0 + p.mt, u.len);
        int c0 = 0, c1 = 0, parts0 = 0, parts1 = 0, ents = 0;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int lo = t0 + (sliced ? 0 : w * a.tt), hi = sliced ? t_end : min(lo + a.tt, t_end);
          if (lo >= t_end) continue;
          const int bound = entry_bound(a, u, hi - 1);
          // with many tokens a list with gaps may hold many chunks that this token does not see yet
          const int seen = a.T > kTileKeys ? entries_up_to(a.union_idx + list, bound, (u.start + hi - 1) >> a.cs_log, lane) : bound;
          const int n = max(0, min(((seen << a.cs_log) + kTileKeys - 1) / kTileKeys, j1) - j0);
          ents = max(ents, seen);
          int c, parts;
          if (sliced) {
            c = w == 0 ? (n + 1) / 2 : n / 2;
            parts = w == 0 ? n_cut : 0;                     // (stream 0 writes for both)
          } else {
            c = n;
            const int mine_cut = n_cut > 1 ? ceil_div(tiles_of(a, bound), cut) : 1;
            parts = j0 < mine_cut * cut ? mine_cut : 0;
          }
          if (w) c1 = c, parts1 = parts;
          else c0 = c, parts0 = parts;
        }
        if (lane == 0) {
          it.unit = unit, it.b = unit / a.Hkv, it.h0 = (unit - it.b * a.Hkv) * a.G, it.t0 = t0, it.start = u.start, it.len = u.len;
          it.j0 = j0, it.ents = ents;
          it.pos_max = u.start + t_end - 1, it.pos_min = u.start + t0;
          it.c[0] = c0, it.c[1] = c1, it.parts[0] = parts0, it.parts[1] = parts1;
          it.part0 = part0, it.part = part, it.cut = cut_no;
          mbar_arrive(item_full + 8 * slot);
        }
        ++n_item;
        if (n_cut > 1) tasks += 2;

      // K's tiles; a batch of 32 entries is loaded while the tiles before it are asked for
        const int nt = sliced ? c0 + c1 : max(c0, c1);
        const int per = 32 / chunks, pos_max = u.start + t_end - 1, pos_min = u.start + t0;
        auto batch = [&](int j) {
          const int e = (j0 + j) * chunks + lane;
          if (e >= ents) return Entry{0, INT_MAX};
          if (a.union_idx[list + e] > pos_max >> a.cs_log) return Entry{0, INT_MAX};     // not seen, not looked at
          return load_entry(a, list, e, ents, staged);
        };
        Entry now = batch(0);
        for (int j = 0; ok && j < nt; j += per) {
          Entry then = {0, INT_MAX};
          if (j + per < nt) then = batch(j + per);
          const uint32_t whole = __ballot_sync(0xffffffffu, now.pos != INT_MAX && now.pos <= pos_min - (a.cs - 1));
          for (int i = 0; i < per && j + i < nt; ++i, ++kt) {
            const uint32_t st = kt % kK;
            if (kt >= kK) ok = wait_warp(k_free + 8 * st, kt / kK - 1);
            if (!ok) break;
            const int sl = __shfl_sync(0xffffffffu, now.slot, i * chunks + ((lane >> 1) & (chunks - 1)));
            const int pos = __shfl_sync(0xffffffffu, now.pos, i * chunks + ((lane >> 1) & (chunks - 1)));
            if (lane < 2 * chunks && (lane & 1) == 0) x.pos[kt % kInfo][lane >> 1] = pos;
            if (lane == 0) {
              const uint32_t all = (1u << chunks) - 1u;
              x.whole[kt % kInfo] = ((whole >> (i * chunks)) & all) == all;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(k_full + 8 * st, kTileBytes);
            __syncwarp();
            if (lane < 2 * chunks) {
                load_chunk(p.k, p.kst, a, sl, pos, lane & 1, k0 + st * kTileBytes + (lane >> 1) * a.cs * 128, k_full + 8 * st);
            }
          }
          now = then;
        }
        if (!sliced) want = __shfl_sync(0xffffffffu, ticket, 0) + cta;
      }
      // copies in flight are waited for before the CTA leaves
      for (uint32_t i = kt >= kK ? kt - kK : 0; i < kt; ++i) mbar_wait(k_full + 8 * (i % kK), (i / kK) & 1u, a.raised);
    } else if (warp == 10) {
      // ------------------------------------------------------------- Q's and V's tiles
      const int64_t staged = staged_slots(a);
      uint32_t vt = 0, nq = 0;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        ok = wait_warp(item_full + 8 * (n & 1u), n >> 1);
        if (!ok) break;
        const Item &it = x.item[n & 1u];
        const int unit = it.unit;
        if (unit < 0) break;
        const int nt = kPairs == 2 ? max(it.c[0], it.c[1]) : it.c[0] + it.c[1];
        const int64_t list = (int64_t)unit * a.umax;
        const int j0 = it.j0, ents = it.ents, pos_max = it.pos_max, pos_min = it.pos_min;
        const bool two = kPairs == 2 && it.c[1] > 0;
        auto batch = [&](int j) {
          const int e = (j0 + j) * chunks + lane;
          if (e >= ents) return Entry{0, INT_MAX};
          if (a.union_idx[list + e] > pos_max >> a.cs_log) return Entry{0, INT_MAX};
          return load_entry(a, list, e, ents, staged);
        };
        Entry now = batch(0);
        if (nt > 0) {
          if (nq > 0) ok = wait_warp(q_free, nq - 1);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(q_full, (uint32_t)(rows_tile * 256 * (two ? 2 : 1)));
          __syncwarp();
          if (lane < (two ? 4 : 2))
            tma_load_4d(q0 + (lane >> 1) * kTileBytes + (lane & 1) * kTileHalfBytes, &p.q, 64 * (lane & 1),
                        it.h0, it.t0 + (lane >> 1) * a.tt, it.b, q_full);
          ++nq;
        }
        const int per = 32 / chunks;
        for (int j = 0; ok && j < nt; j += per) {
          Entry then = {0, INT_MAX};
          if (j + per < nt) then = batch(j + per);
          const uint32_t whole = __ballot_sync(0xffffffffu, now.pos != INT_MAX && now.pos <= pos_min - (a.cs - 1));
          for (int i = 0; i < per && j + i < nt; ++i, ++vt) {
            const uint32_t st = vt % kV;
            if (vt >= kV) ok = wait_warp(v_free + 8 * st, vt / kV - 1);
            if (!ok) break;
            const int sl = __shfl_sync(0xffffffffu, now.slot, i * chunks + ((lane >> 1) & (chunks - 1)));
            const int pos = __shfl_sync(0xffffffffu, now.pos, i * chunks + ((lane >> 1) & (chunks - 1)));
            if (lane < 2 * chunks && (lane & 1) == 0) x.vpos[st][lane >> 1] = pos;
            if (lane == 0) {
              const uint32_t all = (1u << chunks) - 1u;
              x.vwhole[st] = ((whole >> (i * chunks)) & all) == all;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(v_full + 8 * st, kTileBytes);
            __syncwarp();
            if (lane < 2 * chunks) {
              load_chunk(p.v, p.vst, a, sl, pos, lane & 1, v0 + st * kTileBytes + (lane >> 1) * a.cs * 128, v_full + 8 * st);
            }
          }
          now = then;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(item_free + 8 * (n & 1u));
      }
      for (uint32_t i = vt >= kV ? vt - kV : 0; i < vt; ++i) mbar_wait(v_full + 8 * (i % kV), (i / kV) & 1u, a.raised);
      if (nq > 0) mbar_wait(q_full, (nq - 1) & 1u, a.raised);
    } else if (warp == 8) {
      // -------------------------------------------------------------------- products
      // (the whole warp waits and counts, so that what the products are told is uniform)
      constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, 128, 0, 1);
      const uint64_t q_desc = smem_desc_sw128(q0, 16, 1024), k_desc = smem_desc_sw128(k0, 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(v0, kTileHalfBytes, 1024);
      uint32_t t_base = 0, nq = 0, np[2] = {0, 0};
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        ok = wait_warp(item_full + 8 * (n & 1u), n >> 1);
        if (!ok) break;
        const Item &it = x.item[n & 1u];
        if (it.unit < 0) break;
        const int c0 = it.c[0], c1 = it.c[1], steps = max(c0, c1);
        const int nt = kPairs == 2 ? steps : c0 + c1;
        if (nt > 0) ok = wait_warp(q_full, nq++);
        for (int i = 0; ok && i <= steps && nt > 0; ++i) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int cw = w ? c1 : c0;
            if (!ok) break;
            if (i > 0 && i - 1 < cw) {
              const int tile = kPairs == 2 ? i - 1 : 2 * (i - 1) + w;
              const uint32_t t = t_base + tile, st = t % kV;
              ok = wait_warp(v_ok + 8 * st, t / kV);
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                // the weights of 64 keys, then those of the others
                ok = ok && wait_warp((half ? p_ready : p_half) + 8 * w, np[w]);
                if (!ok) break;
                tc_fence_after();
                if (elect_lane()) {
                  const uint64_t vb = v_desc + st * (kTileBytes / 16);
#pragma unroll
                  for (int ks = 4 * half; ks < 4 * half + 4; ++ks) {
                    tc_mma_ts(tmem + 256 + 128 * w, tmem + 128 * w + 8 * ks, vb + ks * (16 * 128 / 16), id_o,
                              i > 1 || ks > 0);
                    if (kLow)
                      tc_mma_ts(tmem + 256 + 128 * w, tmem + 128 * w + 64 + 8 * ks, vb + ks * (16 * 128 / 16), id_o, 1);
                  }
                  if (half) {
                    if (kPairs == 1 || w == 1 || i - 1 >= c1) tc_commit(v_free + 8 * st);
                    if (i == cw) tc_commit(o_full + 8 * w);
                  }
                }
                __syncwarp();
              }
              ++np[w];
              if (!ok) break;
            }
            if (i < cw) {
              const int tile = kPairs == 2 ? i : 2 * i + w;
              const uint32_t t = t_base + tile, st = t % kK;
              ok = wait_warp(k_full + 8 * st, t / kK);
              if (!ok) break;
              tc_fence_after();
              if (elect_lane()) {
                const uint64_t qb = q_desc + (kPairs == 2 ? w * (kTileBytes / 16) : 0);
                const uint64_t kb = k_desc + st * (kTileBytes / 16);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                  const uint32_t off = ((ks >> 2) * kTileHalfBytes + (ks & 3) * 32) / 16;
                  tc_mma(tmem + 128 * w, qb + off, kb + off, id_s, ks > 0);
                }
                mbar_arrive(s_full + 8 * w);     // (hands on the tile's record, which came with K)
                tc_commit(s_full + 8 * w);
                if (kPairs == 1 || w == 1 || i >= c1) tc_commit(k_free + 8 * st);
                if (tile == nt - 1 && (kPairs == 1 || w == 1 || i >= c1)) tc_commit(q_free);
              }
              __syncwarp();
            }
          }
        }
        t_base += nt;
        if (lane == 0) mbar_arrive(item_free + 8 * (n & 1u));
      }
      // every product issued is done before the tensor memory is freed
      if (elect_lane()) tc_commit(mma_done);
      __syncwarp();
      mbar_wait(mma_done, 0, a.raised);
    } else if (warp == 11) {
      // -------------------------------------------- V's tiles that are not seen whole
      uint32_t vt = 0;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        ok = wait_warp(item_full + 8 * (n & 1u), n >> 1);
        if (!ok) break;
        const Item &it = x.item[n & 1u];
        if (it.unit < 0) break;
        const int nt = kPairs == 2 ? max(it.c[0], it.c[1]) : it.c[0] + it.c[1];
        bool found = false;
        for (int j = 0; ok && j < nt; ++j, ++vt) {
          const uint32_t st = vt % kV;
          ok = wait_warp(v_full + 8 * st, vt / kV);
          if (!ok) break;
          if (!x.vwhole[st]) {
            const uint32_t tile = v0 + st * kTileBytes + lane * 16;
            bool fixed = false;
            for (int e0 = 0; e0 < kTileBytes / 16; e0 += 256) {
              // eight pieces a lane: 0 times a finite value is 0, whatever its sign
              uint32_t zero[4] = {0u, 0u, 0u, 0u};
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                uint32_t w[4];
                lds128(tile + (e0 + 32 * k) * 16, w);
#pragma unroll
                for (int q = 0; q < 4; ++q) zero[q] = fma_bf16x2(w[q], 0u, zero[q]);
              }
              if (!__any_sync(0xffffffffu, (zero[0] | zero[1] | zero[2] | zero[3]) != 0u)) continue;
              if (!found) {
                // the records are the item's: the one before has used its own
                found = true;
                if (n > 0) ok = wait_warp(item_free + 8 * ((n - 1) & 1u), (n - 1) >> 1);
                for (int k = lane; k < 3 * 128; k += 32) (&x.bad[0][0])[k] = INT_MAX;
                if (lane == 0) x.bad_item = (int)n;
                __syncwarp();
              }
              fixed = true;
#pragma unroll 1
              for (int e = e0 + lane; e < e0 + 256; e += 32) {
                const uint32_t at = v0 + st * kTileBytes + e * 16;
                uint32_t w[4];
                lds128(at, w);
                const int row = (e & 1023) >> 3, col0 = (e >> 10) * 64 + (((e & 7) ^ (row & 7)) << 3);
                const int first = x.vpos[st][row >> a.cs_log], pos = first == INT_MAX ? INT_MAX : first + (row & (a.cs - 1));
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const uint32_t v = (w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
                  if ((v & 0x7F80u) == 0x7F80u) {
                    const int kind = (v & 0x7Fu) ? 0 : ((v & 0x8000u) ? 2 : 1);
                    atomicMin(&x.bad[kind][col0 + k], pos);
                    w[k >> 1] &= (k & 1) ? 0x0000FFFFu : 0xFFFF0000u;
                  }
                }
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
              }
            }
            if (fixed)
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(v_ok + 8 * st);
        }
        __syncwarp();
        if (lane == 0) {
          __threadfence_block();
          mbar_arrive(looked + 8 * (n & 1u));
          mbar_arrive(item_free + 8 * (n & 1u));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------------- softmax
    const int w = warp >> 2, quarter = warp & 3, r = 32 * quarter + lane;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_at = tmem + lane_base + 128 * w, o_at = tmem + lane_base + 256 + 128 * w;
    const int tok = r / a.G, head = r % a.G;
    const bool some = 32 * quarter < rows_tile;            // of this warp's rows are query rows
    uint32_t ns = 0, no = 0, n_both = 0, n_parts = 0, t_base = 0;
    // (one row tile leaves the second's queries' place free, few rows their own tile's later ones)
    float2 *stat = reinterpret_cast<float2 *>(smem + (kLow ? 64 * 128 : kTileBytes));
    bool ok = true;
    for (uint32_t n = 0; ok && !pending; ++n) {
      ok = wait_warp(item_full + 8 * (n & 1u), n >> 1);
      if (!ok) break;
      const Item &it = x.item[n & 1u];
      const int unit = it.unit;
      if (unit < 0) break;
      const int cw = it.c[w], parts = it.parts[w];
      const int nt = kPairs == 2 ? max(it.c[0], it.c[1]) : it.c[0] + it.c[1];
      const int token = it.t0 + (kPairs == 2 ? w * a.tt : 0) + tok;
      const bool valid = r < rows_tile && token < it.len;
      const int pos = valid ? it.start + token : -1;
      float m = -INFINITY, l = 0.f;                        // reference (a score before the factor), sum of weights
      float sub = 0.f;                                     // the reference times the factor, negated
      bool far = false;
      for (int i = 0; i < cw; ++i) {
        const uint32_t t = t_base + (kPairs == 2 ? i : 2 * i + w);
        ok = wait_warp(s_full + 8 * w, ns);
        ++ns;
        if (!ok) break;
        tc_fence_after();
        if (some) {
          const int whole = x.whole[t % kInfo];
          float s[128];
          // the second half is on its way while the first is looked over
          tmem_ld32(s_at, s), tmem_ld32(s_at + 32, s + 32);
          tmem_wait_ld();
          tmem_ready(s), tmem_ready(s + 32);
          tmem_ld32(s_at + 64, s + 64), tmem_ld32(s_at + 96, s + 96);
          float mx = -INFINITY;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half) {
              tmem_wait_ld();
              tmem_ready(s + 64), tmem_ready(s + 96);
            }
            if (!whole) {
#pragma unroll
              for (int h = 4 * half; h < 4 * half + 4; ++h) {
                const int row0 = 16 * h, first = x.pos[t % kInfo][row0 >> a.cs_log];
                // columns up to `lim` are seen
                const int lim = first == INT_MAX ? -1 : pos - first - (row0 & (a.cs - 1));
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (e > lim) s[16 * h + e] = -INFINITY;
              }
            }
            float m4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(s[64 * half + e], s[64 * half + 4 + e]);
#pragma unroll
            for (int h = 8; h < 64; h += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], s[64 * half + h + e], s[64 * half + h + 4 + e]);
            mx = max3(mx, max3(m4[0], m4[1], m4[2]), m4[3]);
          }
          // (also from -inf; not where both are; rows that are none hold anything and have no say)
          const bool up = valid && (mx - m) * a.sl2 > kHead;
          if (__any_sync(0xffffffffu, up)) {
            const float f = up ? ex2_approx((m - mx) * a.sl2) : 1.f;
            if (up) m = mx;
            l *= f;
            if (i > 0) {
              // S(t) is there, so the product before it is done with O
#pragma unroll 1
              for (int h = 0; h < 4; ++h) {
                float o[32];
                tmem_ld32(o_at + 32 * h, o);
                tmem_wait_ld();
                tmem_ready(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st32(o_at + 32 * h, o);
              }
              tmem_wait_st();
            }
            // weights are 2^(s sl2 - m sl2), one rounding of a number near 0 or of one that gives no weight; scores
            // so large that m sl2 itself is rounded by more than 2^-8 are taken from the reference first
            sub = m == -INFINITY ? 0.f : -m * a.sl2;
            far = __any_sync(0xffffffffu, valid && !(fabsf(sub) <= 65536.f));
          }
          float add = sub;
          if (far) {
#pragma unroll
            for (int e = 0; e < 128; ++e) s[e] -= m == -INFINITY ? 0.f : m;
            add = 0.f;
          }
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[16], low[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 y = fma2(make_float2(s[32 * h + 2 * e], s[32 * h + 2 * e + 1]), make_float2(a.sl2, a.sl2),
                              make_float2(add, add));
              y.x = ex2_approx(y.x), y.y = ex2_approx(y.y);
              sum[e & 1] = add2(sum[e & 1], y);
              if (!kLow) {
                pk[e] = cvt_bf16x2(y.x, y.y);
              } else {
                // the upper 16 bits, and what is left: never negative, and above 0 where the weight is, so that an
                // infinity of V stays one
                const uint32_t a0 = __float_as_uint(y.x), a1 = __float_as_uint(y.y);
                pk[e] = __byte_perm(a0, a1, 0x7632);
                const float2 cut = make_float2(-__uint_as_float(a0 & 0xFFFF0000u), -__uint_as_float(a1 & 0xFFFF0000u));
                const float2 rest = fma2(y, make_float2(0x1p-20f, 0x1p-20f), add2(y, cut));
                low[e] = cvt_bf16x2(rest.x, rest.y);
              }
            }
            tmem_st16(s_at + 16 * h, pk);
            if (kLow) tmem_st16(s_at + 64 + 16 * h, low);
            if (h == 1) {
              // the first 64 keys' product may begin
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(p_half + 8 * w);
            }
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_wait_st();
        } else if (lane == 0) {
          mbar_arrive(p_half + 8 * w);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + 8 * w);
      }
      if (!ok) break;
      t_base += nt;

      // ------------------------------------------------------------ the item's sums
      ok = wait_warp(looked + 8 * (n & 1u), n >> 1);
      if (!ok) break;
      if (cw > 0) {
        ok = wait_warp(o_full + 8 * w, no++);
        if (!ok) break;
        tc_fence_after();
      }
      const bool both = kPairs == 1 && it.c[1] > 0;       // the streams have sums of the same rows
      if (both && w == 1) {
        // stream 0 takes O out of this one's columns: it has the same lanes
        stat[r] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(handed);
        ok = wait_warp(taken, n_both++);
        if (!ok) break;
      } else if (parts > 0) {
        float f0 = 1.f, f1 = 0.f;
        if (both) {
          ok = wait_warp(handed, n_both++);
          if (!ok) break;
          tc_fence_after();
          const float2 other = stat[r];
          const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
          f0 = ex2_approx((m - ref) * a.sl2), f1 = ex2_approx((other.x - ref) * a.sl2);
          m = top, l = l * f0 + other.y * f1;
        }
        const int b = it.b, h0 = it.h0;
        const int64_t slot = it.part + (kPairs == 2 ? w : 0);
        float *po = p.part_o + (slot * rows_tile + r) * kD;
        const int64_t row = ((int64_t)b * a.T + token) * a.Hq + h0 + head;
        uint16_t *dst = p.out + b * p.os[0] + token * p.os[1] + (h0 + head) * p.os[2];
        if (parts == 1) f0 = l == 0.f ? 0.f : f0 / l, f1 = l == 0.f ? 0.f : f1 / l;
        if (some) {
          const bool none = cw == 0 || l == 0.f;
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            float o[32];
            if (cw > 0) {
              tmem_ld32(o_at + 32 * h, o);
              tmem_wait_ld();
              tmem_ready(o);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * f0;
            if (both) {
              float o1[32];
              tmem_ld32(o_at + 128 + 32 * h, o1);
              tmem_wait_ld();
              tmem_ready(o1);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : fmaf(o1[e], f1, o[e]);
            }
            if (valid) {
              if (parts == 1) {
                uint32_t v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = cvt_bf16x2(o[2 * e], o[2 * e + 1]);
                if (p.wide) {
                  store32(dst + 32 * h, v), store32(dst + 32 * h + 16, v + 8);
                } else {
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<uint4 *>(dst + 32 * h + 8 * e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) store32(po + 32 * h + 8 * e, reinterpret_cast<const uint32_t *>(o) + 8 * e);
              }
            }
          }
          if (valid && x.bad_item == (int)n) {
            // values of V that were taken out of a tile, where the row sees them
#pragma unroll 1
            for (int c = 0; c < 128; ++c) {
              const bool nan = x.bad[0][c] <= pos, up = x.bad[1][c] <= pos, down = x.bad[2][c] <= pos;
              if (!nan && !up && !down) continue;
              const float add = nan || (up && down) ? NAN : (up ? INFINITY : -INFINITY);
              if (parts == 1) dst[c] = (uint16_t)f2bf(bf_lo(dst[c]) + add);
              else po[c] += add;
            }
          }
          if (valid) {
            if (parts == 1) {
              if (p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m == -INFINITY ? NAN : m * a.scale + logf(l));
            } else {
              p.part_ml[slot * rows_tile + r] = make_float2(m, l);
            }
          }
        }
        if (both) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(taken);
        }
        if (parts > 1) {
          // (a wait that gives up: a warp may have done so already, before an event that the others still saw)
          __syncwarp();
          if (lane == 0) mbar_arrive(stored + 8 * w);
          ok = wait_warp(stored + 8 * w, n_parts++);
          if (!ok) break;
          if (quarter == 0 && lane == 0) {
            __threadfence();
            int32_t *ctr = p.w.ctr + 2 + it.cut + (kPairs == 2 ? w : 0);
            if (atomicAdd(ctr, 1) == parts - 1) {
              // the last part: joined when the CTA is through with its items
              *ctr = 0;
              Task &k = x.task[atomicAdd(&x.tasks, 1)];
              k.unit = unit, k.len = it.len, k.token = it.t0 + (kPairs == 2 ? w * a.tt : 0);
              k.parts = parts, k.first = it.part0 + (kPairs == 2 ? w : 0);
            }
            __threadfence();
          }
        }
      }
      tc_fence_before();          // O is read before the next item's first product overwrites it
      __syncwarp();
      if (lane == 0) mbar_arrive(item_free + 8 * (n & 1u));
    }
    // ------------------------------------------------- row tiles whose last part came from here
    asm volatile("bar.sync 3, 256;" ::: "memory");
    const int tasks = *(volatile int *)&x.tasks;
    for (int k = 0; k < tasks; ++k) {
      const Task &task = x.task[k];
      const int b = task.unit / a.Hkv, h0 = task.unit % a.Hkv * a.G;
      Join q;
      q.part_o = p.part_o, q.part_ml = p.part_ml, q.first = task.first, q.pairs = kPairs, q.parts = task.parts;
      q.rows = min(rows_tile, (task.len - task.token) * a.G), q.rows_tile = rows_tile, q.G = a.G, q.Hq = a.Hq;
      q.scale = a.scale, q.sl2 = a.sl2;
      q.out = p.out + b * p.os[0] + task.token * p.os[1] + h0 * p.os[2], q.os1 = p.os[1], q.os2 = p.os[2];
      q.lse = p.lse ? p.lse + ((int64_t)b * a.T + task.token) * a.Hq + h0 : nullptr;
      // (few rows have many parts: one warp a row)
      if (q.rows <= 32) join_rows<1, 16>(q, warp, 8);
      else if (q.parts <= 4) join_rows<4, 4>(q, warp, 8);
      else join_rows<2, 8>(q, warp, 8);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
  }
  leave_counters(p.w, a, &x.pending);
}

struct Shape {
  int tt, pairs, mt, rows;
  int64_t slots;
};

Shape shape_of(int T, int G, int cta) {
  Shape s;
  s.tt = T < 128 / G ? T : 128 / G;
  s.pairs = T > s.tt ? 2 : 1;
  s.mt = s.pairs * s.tt;
  s.rows = s.tt * G;
  s.slots = (s.pairs == 1 ? 2 : 10) * (int64_t)cta;    // parts: 2 a slice, 2 a range of a pair
  return s;
}

}  // namespace

int64_t extend_workspace(int B, int T, int Hq, int Hkv, int sm_count) {
  if (B == 0 || T == 0) return 0;
  const Shape s = shape_of(T, Hq / Hkv, sm_count);
  return s.slots * s.rows * (kD + 2) * 4;
}

cudaError_t launch_extend(const ExtendArgs &e, cudaStream_t stream) {
  const PagesArgs &a = e.p;
  const Shape s = shape_of(a.T, a.G, e.sm_count);
  ExtendParams p{};
  p.a = a;
  p.a.tt = s.tt;
  const bool hot = a.hot_slots > 0, far = a.max_misses > 0;
  if (!make_rows_map(&p.q, e.q, e.q_stride, a.B, a.T, a.Hq, a.G, s.tt) ||
      !make_pages_map(&p.k, hot ? e.Khot : e.dummy, hot ? a.hot_slots : 1, a.cs) ||
      !make_pages_map(&p.v, hot ? e.Vhot : e.dummy, hot ? a.hot_slots : 1, a.cs) ||
      !make_pages_map(&p.kst, far ? e.Kst : e.dummy, far ? a.max_misses : 1, a.cs) ||
      !make_pages_map(&p.vst, far ? e.Vst : e.dummy, far ? a.max_misses : 1, a.cs))
    return cudaErrorInvalidValue;
  p.out = static_cast<uint16_t *>(e.out);
  for (int i = 0; i < 3; ++i) p.os[i] = e.out_stride[i];
  p.lse = e.lse;
  p.wide = reinterpret_cast<uintptr_t>(e.out) % 32 == 0 && e.out_stride[0] % 16 == 0 && e.out_stride[1] % 16 == 0 &&
           e.out_stride[2] % 16 == 0;
  p.part_o = e.parts;
  p.part_ml = reinterpret_cast<float2 *>(e.parts + s.slots * s.rows * kD);
  p.w = {e.ctr, kCtrPerCta * e.sm_count};
  p.mt = s.mt;
  auto *kernel = s.pairs == 2 ? &k_extend<2, false> : (s.rows <= kLowRows ? &k_extend<1, true> : &k_extend<1, false>);
  const cudaError_t r = set_dyn_smem((const void *)kernel, kSmem);
  if (r != cudaSuccess) return r;
  return launch_k(kernel, dim3(e.sm_count), dim3(kThreads), kSmem, stream, p);
}

}  // namespace dd
