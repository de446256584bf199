// Shared device code of the two attentions over 4-bit pages (dd_attn4.cu: mma.sync, up to
// 16 query vectors a unit; dd_attn4_tc.cu: tcgen05, up to 64): the units and how the CTAs share
// them, the blocks' look-up and loads, the queries in fp16, the step's own rows and the
// joining of a unit's parts.
#pragma once

#include <float.h>
#include <limits.h>

#include "dd_attn.cuh"
#include "dd_kv4.cuh"
#include "dd_tc.cuh"

namespace dd {

constexpr int kMaxRuns = 16;             // units of a slice listed at a time
constexpr float kLazy = 8.f;             // a score may exceed the reference by 2^kLazy ...
constexpr float kHead = 6.f;             // ... and weights are held times 2^kHead

// The highest score that leaves reference m in place.  Rounded down, as from 2^25 on floats are 4 apart
// and the nearest one may lie above m + 14: no float is left out between this one and the sum.
__device__ __forceinline__ float highest_for(float m) { return __fadd_rd(m, kLazy + kHead); }

struct Run {           // a unit's place in the sequence of tiles
  int unit, b, g;                  // unit, request, KV head
  int start, end, cnt, len;        // tiles [start, end) of the sequence; chunks; rows (INT_MAX: no kv_len)
  int cta0, cta1;                  // the CTAs that share it
  int ke, ve;
};

struct Attn4Params {
  Attn4Args a;
  int NQ, G, bpc_shift, group_q, units;    // group_q: query vectors of a part (NQ rounded up to 8)
  float *part_o, *part_ml;
  int32_t *arrive;
};

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// shared-memory loads by address (asm: the ring is written by bulk copies)
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(p));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(p));
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t p) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(p));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t p) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(p));
  return r;
}

// Tiles of a unit: its union's blocks of 16 rows, 2^tile_shift a tile, those wholly
// behind the end left out (chunk numbers ascend, so block x lies at position 16 x or
// later), at least one tile, so that a unit without rows is visited too.
struct Lengths {
  int cnt, len, exps;      // chunks, rows (INT_MAX without kv_len), ke | ve << 16
};
__device__ __forceinline__ int unit_tiles(const Attn4Params &p, int unit, int tile_shift, Lengths &r) {
  const Attn4Args &a = p.a;
  const int b = unit / a.Hkv, g = unit - b * a.Hkv;
  r.cnt = a.union_cnt[unit];
  r.len = a.kv_len ? a.kv_len[b] : INT_MAX;
  int ke = a.k_exp ? a.k_exp[g] : 0;
  int ve = a.v_exp ? a.v_exp[g] : 0;
  if (r.cnt < 0 || r.cnt > a.umax || abs(ke) > kMaxExp4 || abs(ve) > kMaxExp4) {
    set_status(a.status, DD_ERR_DEVICE_CHECK);
    r.cnt = r.cnt < 0 ? 0 : min(r.cnt, a.umax);
    ke = max(-kMaxExp4, min(ke, kMaxExp4));
    ve = max(-kMaxExp4, min(ve, kMaxExp4));
  }
  r.exps = (ke & 0xFFFF) | ve << 16;
  r.len = max(r.len, 0);
  const int n = min(r.cnt << p.bpc_shift, (r.len >> 4) + ((r.len & 15) != 0));
  return max((n + (1 << tile_shift) - 1) >> tile_shift, 1);
}

__device__ __forceinline__ void fill_run(const Attn4Params &p, Run &r, int unit, int start, int end,
                                         const Lengths &l) {
  r.unit = unit;
  r.b = r.unit / p.a.Hkv;
  r.g = r.unit - r.b * p.a.Hkv;
  r.start = start;
  r.end = end;
  r.cnt = l.cnt;
  r.len = l.len;
  r.ke = (int)(int16_t)(l.exps & 0xFFFF);
  r.ve = l.exps >> 16;
}

// 2^(a - b) with equal arguments (both -inf among them) giving 1
__device__ __forceinline__ float weight_of(float a, float b) { return a == b ? 1.f : exp2f(a - b); }

// Four columns of a query vector's sums with their reference and weight sum.
struct Part {
  float m, l;
  float4 o;
};

__device__ __forceinline__ int64_t out_row(const Attn4Params &p, int unit, int qv) {   // of q and out, in elements
  const int b = unit / p.a.Hkv, g = unit - b * p.a.Hkv, j = qv / p.G, h = g * p.G + qv - j * p.G;
  return ((int64_t)(b * p.a.n_q + j) * p.a.Hq + h) * kD;
}

// Step's own rows (in shared memory: keys, then values), then the division.  The lane
// holds columns 4 lane .. of the query vector (qw).
__device__ __forceinline__ void finish(const Attn4Params &p, int unit, int qv, Part s, uint2 qw, const uint2 *tails,
                                       int lane) {
  const Attn4Args &a = p.a;
  if (a.k_tail) {
    const float sl2 = a.softmax_scale * 1.4426950408889634f;
    const int j = qv / p.G;
    for (int t = 0; t <= j; ++t) {
      const uint2 kw = tails[t * 32 + lane], vw = tails[(kMaxNq + t) * 32 + lane];
      float x = bf_lo(qw.x) * bf_lo(kw.x);
      x = fmaf(bf_hi(qw.x), bf_hi(kw.x), x);
      x = fmaf(bf_lo(qw.y), bf_lo(kw.y), x);
      x = fmaf(bf_hi(qw.y), bf_hi(kw.y), x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      x *= sl2;
      const float m = fmaxf(s.m, x);      // a NaN score leaves m: its weight is NaN, ...
      const float wa = weight_of(s.m, m), wt = exp2f(x - m);      // ... as is that of +inf, and of -inf alone
      s.l = s.l * wa + wt;
      s.o.x = s.o.x * wa + wt * bf_lo(vw.x);
      s.o.y = s.o.y * wa + wt * bf_hi(vw.x);
      s.o.z = s.o.z * wa + wt * bf_lo(vw.y);
      s.o.w = s.o.w * wa + wt * bf_hi(vw.y);
      s.m = m;
    }
  }
  // no row at all: zeros (a NaN is kept)
  const float4 r = s.l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : make_float4(s.o.x / s.l, s.o.y / s.l, s.o.z / s.l, s.o.w / s.l);
  *reinterpret_cast<float4 *>(a.out + out_row(p, unit, qv) + 4 * lane) = r;
}

// 32 query values of a lane as fp16 pairs, scaled by a power of two so that the largest of
// the 128 values of the query vector (four neighbouring lanes) lies just below 2^15, and
// the factor back (lanes: those that take part).
__device__ __forceinline__ void query_fragments(const uint4 (&w)[4], uint32_t (&f)[16], float &back, unsigned lanes = 0xFFFFFFFFu) {
  const uint32_t v[16] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w,
                          w[2].x, w[2].y, w[2].z, w[2].w, w[3].x, w[3].y, w[3].z, w[3].w};
  uint32_t top = 0;   // largest magnitude, as bits
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, max((v[i] & 0x7FFFu) << 16, v[i] & 0x7FFF0000u));
  top = max(top, __shfl_xor_sync(lanes, top, 1));
  top = max(top, __shfl_xor_sync(lanes, top, 2));
  // beside an infinite (or NaN) value every finite one stays finite: what it adds does not matter,
  // an infinity of its own would
  const int e = min((int)(top >> 23), 254);
  const int sh = top == 0 ? 0 : min(126, 14 - (e - 127));
  const float mul = pow2i(sh);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = cvt_f16x2(bf_lo(v[i]) * mul, bf_hi(v[i]) * mul);
  back = pow2i(-sh);
}

// From a product of scaled queries to a score, finite: a product of 0 stays a score of 0.
// (Where this passes fp32, products differ by 2^-34 at least, so scores by 2^94: one row has all the
// weight either way.)
__device__ __forceinline__ float score_factor(float back, float kmul) { return fminf(back * kmul, FLT_MAX); }

// The unit's own new rows into shared memory (keys, then values, 16 pieces a row), by
// asynchronous copies of `threads` threads.
__device__ __forceinline__ void stage_tails(const Attn4Params &p, const Run &r, uint4 *s_tails, int tid, int threads) {
  const Attn4Args &a = p.a;
  if (!a.k_tail) return;
  for (int i = tid; i < 2 * a.n_q * 16; i += threads) {
    const int kv = i >= a.n_q * 16, e = kv ? i - a.n_q * 16 : i;
    const uint16_t *src = static_cast<const uint16_t *>(kv ? a.v_tail : a.k_tail);
    cp_async16(s_tails + kv * kMaxNq * 16 + e, reinterpret_cast<const uint4 *>(
        src + ((int64_t)(r.b * a.n_q + (e >> 4)) * a.Hkv + r.g) * kD) + (e & 15));
  }
}

// Block `blk` of a run: its slot, and {query mask, rows in use << 8, block of the chunk <<
// 13}, 0 where no query sees a row of it.
struct BlockRef {
  int slot;
  uint32_t meta;
};
// (The union's entry is loaded first and looked at later, so that other work fits in between.)
struct Entry {
  int slot, idx, sub, len;       // sub: block of the chunk, -1: no such block
  uint32_t qm;
};
__device__ __forceinline__ Entry load_entry(const Attn4Params &p, const Run &r, int blk, uint32_t all_q) {
  const Attn4Args &a = p.a;
  const int ci = blk >> p.bpc_shift;
  Entry n = {0, 0, -1, r.len, all_q};
  if (ci < r.cnt) {
    const int64_t e = (int64_t)r.unit * a.umax + ci;
    n.sub = blk & ((1 << p.bpc_shift) - 1);
    n.slot = a.union_slot[e];
    if (a.union_qmask) n.qm = a.union_qmask[e];
    if (a.kv_len) n.idx = a.union_idx[e];
  }
  return n;
}
__device__ __forceinline__ BlockRef look_at(const Attn4Params &p, const Entry &n, int64_t staged, uint32_t all_q) {
  const Attn4Args &a = p.a;
  if (n.sub < 0) return {0, 0u};
  const int slot = n.slot, sub = n.sub;
  const uint32_t qm = n.qm & all_q;
  int rows = 16;
  if (a.kv_len) {
    const int64_t left = n.len - ((int64_t)n.idx * a.cs + sub * 16);
    rows = left < 0 ? 0 : left > 16 ? 16 : (int)left;
  }
  uint32_t meta = qm && rows ? qm | (uint32_t)rows << 8 | (uint32_t)sub << 13 : 0u;
  // (whatever the tiles' size: only a slot that is going to be read has to be one)
  if (meta && (slot >= 0 ? slot >= a.hot_slots : -1 - (int64_t)slot >= staged)) {
    set_status(a.status, DD_ERR_DEVICE_CHECK);
    meta = 0u;
  }
  return {slot, meta};
}

// K and V of a block into shared memory (K first), completing on bar.
__device__ __forceinline__ void load_block(const Attn4Params &p, const BlockRef &r, uint32_t dst, uint32_t bar) {
  const Attn4Args &a = p.a;
  const int64_t page = (int64_t)kBlk4 << p.bpc_shift;
  const int64_t off = (r.slot >= 0 ? (int64_t)r.slot : -1 - (int64_t)r.slot) * page + (int64_t)(r.meta >> 13) * kBlk4;
  mbar_arrive_expect_tx(bar, 2 * kBlk4);
  bulk_load(dst, (r.slot >= 0 ? a.Khot : a.Kst) + off, kBlk4, bar);
  bulk_load(dst + kBlk4, (r.slot >= 0 ? a.Vhot : a.Vst) + off, kBlk4, bar);
}

// The copies of tiles [from, to) of a ring (at most 32, all asked for) have landed, or have had the
// time of one wait to: a CTA does not leave with copies on their way to its shared memory.
// All lanes of a warp.
__device__ __forceinline__ void ring_drain(uint32_t bar0, uint32_t stages, uint32_t from, uint32_t to, int lane,
                                           int32_t *status) {
  const uint32_t t = from + (uint32_t)lane;
  if (t < to) mbar_wait(bar0 + 8 * (t % stages), (t / stages) & 1u, status);
  __syncwarp();
}

// A warp's wait for tile t of its ring (all lanes).  False where it runs out: what is behind it,
// up to tile `last`, is drained, and the warp waits for no other tile.
template <uint32_t S>
__device__ __forceinline__ bool ring_wait(uint32_t bar0, uint32_t t, uint32_t last, int lane, int32_t *status) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * (t % S), (t / S) & 1u, status));
  if (!ok) ring_drain(bar0, S, t + 1, last + 1, lane, status);
  return ok;
}

// One thread: the CTA is done with the run's unit, which others share.  True for the last one
// to come, which then joins the parts, unless one of them did no work (dead: it began after
// an error had been reported, by this call's own CTAs perhaps, and left its part of the
// workspace as an earlier call did): those are counted in the upper half.
__device__ __forceinline__ bool arrive_at_unit(const Attn4Params &p, const Run &r, bool dead) {
  const uint32_t before = (uint32_t)atom_add_acq_rel_gpu(p.arrive + r.unit, dead ? 0x10001 : 1);
  if ((int)(before & 0xFFFFu) != r.cta1 - r.cta0) return false;
  p.arrive[r.unit] = 0;        // for the next call
  return !dead && before < 0x10000u;
}

// Query vector k of the run's group from the parts of all its CTAs.
__device__ __forceinline__ Part combine_parts(const Attn4Params &p, const Run &r, int k, int lane) {
  const int group_q = p.group_q;
  // 32 parts at a time: a lane holds one's reference and weight, the sums of eight are in flight
  Part s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int k0 = r.cta0; k0 <= r.cta1; k0 += 32) {
    const int np = min(32, r.cta1 - k0 + 1);
    const int64_t at0 = ((int64_t)k0 + r.unit) * group_q + k;
    const float4 *src = reinterpret_cast<const float4 *>(p.part_o + at0 * kD) + lane;
    const int64_t step = (int64_t)group_q * (kD / 4);
    float4 v[8];     // on their way while the weights are worked out
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = __ldcg(src + min(t, np - 1) * step);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < np) ml = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + 2 * (at0 + (int64_t)lane * group_q)));
    float mn = fmaxf(s.m, ml.x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
    const float wa = weight_of(s.m, mn), wt = weight_of(ml.x, mn);
    float lw = lane < np ? wt * ml.y : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, d);
    s.l = s.l * wa + lw;
    s.o.x *= wa, s.o.y *= wa, s.o.z *= wa, s.o.w *= wa;
    for (int t0 = 0; t0 < np; t0 += 8) {
      if (t0 > 0) {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = __ldcg(src + min(t0 + t, np - 1) * step);
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float f = __shfl_sync(0xffffffffu, wt, (t0 + t) & 31);
        if (t0 + t < np) {
          s.o.x = fmaf(f, v[t].x, s.o.x);
          s.o.y = fmaf(f, v[t].y, s.o.y);
          s.o.z = fmaf(f, v[t].z, s.o.z);
          s.o.w = fmaf(f, v[t].w, s.o.w);
        }
      }
    }
    s.m = mn;
  }
  return s;
}

// ------------------------------------------------------------- a CTA's slice
struct PlanSmem {
  Run runs[kMaxRuns];
  int scratch[33];
  int first, flag, lo, hi;
};

// Equal slices of the sequence, in whole rounds of the CTA's kQuantum warps.  A slice
// that holds the end of one unit and the start of the next pays for two queries and two
// joins, two to three rounds' time, so where the units are no more than the threads
// (their lengths are then loaded once) and parts of up to two rounds more than a slice
// let every CTA work on one unit, the units are cut into such parts instead.
// Llama-3-8B layer, two queries: 21.0 -> 18.8 us; three requests, 21 units: 32.4 -> 20.8 us.
template <int kThreads, int kQuantum, int kTileShift>
struct Slice {
  Lengths mine{};
  int my_tiles = 0, my_start = 0, total = 0, per = 0, lo = 0, hi = 0;
  int64_t staged = 0;
  bool one_round = false, parts = false, dead = false;

  // All threads.  False: nothing to do for this CTA.
  __device__ __forceinline__ bool open(const Attn4Params &p, PlanSmem &sm) {
    const Attn4Args &a = p.a;
    const int tid = threadIdx.x;
    one_round = p.units <= kThreads;
    // all loads before the first use of one
    const int pending = tid == 0 ? load_status(a.status) : 0;
    const int missing = a.miss_count ? *a.miss_count : INT_MAX;
    if (one_round) {
      if (tid < p.units) my_tiles = unit_tiles(p, tid, kTileShift, mine);
      if (tid == 0) sm.flag = pending;
      my_start = block_excl_scan(my_tiles, sm.scratch, &total);
    } else {
      for (int u = tid; u < p.units; u += kThreads) my_tiles += unit_tiles(p, u, kTileShift, mine);
      if (tid == 0) sm.flag = pending;
      total = block_sum(my_tiles, sm.scratch);
    }
    staged = min((int64_t)missing, a.max_misses);
    dead = sm.flag != 0;       // an error is pending: no work (the arrival counts go on)
    const int n_cta = (int)gridDim.x;
    per = ((total + n_cta - 1) / n_cta + kQuantum - 1) / kQuantum * kQuantum;
    lo = (int)min((int64_t)total, (int64_t)blockIdx.x * per);
    hi = min(total, lo + per);
    if (one_round && n_cta + kThreads < 1024) {
      // the number of parts for three part lengths, 10 bits each (at most n_cta + units)
      constexpr int kStep = kQuantum > 1 ? kQuantum : 4;
      int mine3 = 0, all3;
#pragma unroll
      for (int k = 0; k < 3; ++k) mine3 |= (my_tiles + per + k * kStep - 1) / (per + k * kStep) << (10 * k);
      const int before3 = block_excl_scan(mine3, sm.scratch, &all3);
#pragma unroll
      for (int k = 2; k >= 0; --k) {
        if ((all3 >> (10 * k) & 1023) > n_cta) continue;
        parts = true;
        if (k > 0 && (all3 >> (10 * (k - 1)) & 1023) <= n_cta) continue;      // a shorter one fits
        const int n = mine3 >> (10 * k) & 1023, first = before3 >> (10 * k) & 1023;
        const int part = (int)blockIdx.x - first;
        hi = (int)blockIdx.x < (all3 >> (10 * k) & 1023);           // does this CTA have a part?
        lo = 0;
        if (n && part >= 0 && part < n) {
          const int len = (my_tiles + n - 1) / n;
          fill_run(p, sm.runs[0], tid, my_start, my_start + my_tiles, mine);
          sm.runs[0].cta0 = first;
          sm.runs[0].cta1 = first + n - 1;
          sm.lo = my_start + part * len;
          sm.hi = min(my_start + my_tiles, sm.lo + len);
        }
      }
    }
    return lo < hi;
  }

  // All threads: lists the slice's units number w0 .. w0 + kMaxRuns - 1, of which the slice
  // has tiles wlo .. whi - 1, and returns how many there are.  The slice ends where whi == hi.
  __device__ __forceinline__ int list(const Attn4Params &p, PlanSmem &sm, int w0, int &wlo, int &whi) {
    // for what the list held before, and for the part that open() wrote
    __syncthreads();
    int n_seen = 0;                    // units of the slice seen
    if (parts) {
      n_seen = 1;
      lo = sm.lo;
      hi = sm.hi;
    } else {
      const int tid = threadIdx.x;
      int base = 0;                    // tiles of the units before this round
      for (int u0 = 0; u0 < p.units && base < hi; u0 += kThreads) {
        int all = total, start = my_start;
        if (!one_round) {
          const int u = u0 + tid;
          my_tiles = u < p.units ? unit_tiles(p, u, kTileShift, mine) : 0;
          start = base + block_excl_scan(my_tiles, sm.scratch, &all);
        }
        const bool in = my_tiles && start < hi && start + my_tiles > lo;
        if (in && start <= lo) sm.first = u0 + tid;
        const int n = __syncthreads_count(in);
        if (n) {
          const int rank = u0 + tid - sm.first - w0;
          if (in && rank >= 0 && rank < kMaxRuns) {
            fill_run(p, sm.runs[rank], u0 + tid, start, start + my_tiles, mine);
            sm.runs[rank].cta0 = start / per;
            sm.runs[rank].cta1 = (start + my_tiles - 1) / per;
          }
          n_seen += n;
        }
        base += all;
      }
      __syncthreads();
    }
    const int n_runs = min(n_seen - w0, kMaxRuns);
    wlo = max(lo, sm.runs[0].start);
    whi = min(hi, sm.runs[n_runs - 1].end);
    return n_runs;
  }
};

// dd_attn4_tc.cu: one CTA per SM, tiles of 128 rows, all query vectors of a unit at once
cudaError_t launch_attn4_tc(int grid, const Attn4Params &p, cudaStream_t s);

}  // namespace dd
