// Attention over a cache held in 4 bits: out = softmax(scale q.K^T) V over the rows
// of the union's chunks that each query selected, K and V decoded on the way.
//
// Bytes and issue slots.  A row of K and V is 144 bytes, which HBM brings an SM
// every 6 cycles; its 256 codes have to be decoded in those 24 issue slots of a
// warp (8 values each).  So the codes go from shared memory straight into the
// registers of the matrix instruction that uses them, one conversion and one
// multiplication by the scale per two values, and never back:
//   S^T = K Q^T  (mma m16n8k16, A = 16 rows of K, B = 8 query vectors): a lane
//     takes 32 consecutive values of two rows (one 16-byte load each; the order
//     of the 128 terms of a dot product is free, so Q is laid out to match);
//   O^T += V^T P^T (A = 16 columns of V over 16 rows): the instruction wants two
//     rows' values of a column side by side, so the nibbles of two rows are
//     interleaved before they are converted.
// Query vectors are the narrow side (8 a tile), so the 4 or 8 of a KV head's
// group are not padded to 16.
//
// Precision.  A code times its scale is exact in fp16.  A query vector is scaled
// by a power of two to just below 2^15, where its 8-bit significands are exact in
// fp16 down to 2^-32 of its largest value.  P is split into two fp16 parts (22
// bits).  The matrix unit adds up 32 rows at a time; the running sums are added
// in fp32 outside of it, where additions round to nearest: its own truncates, and
// over the hundreds of additions of a long context that shows (1e-5).
// The softmax's reference value is moved only when a score exceeds it by 2^8, so
// most tiles need no maximum across lanes (P stays below 2^14).
//
// Work split: the unions' tiles of 32 rows (two blocks) of all (request, KV head)
// units, laid end to end, are cut into equal slices, one for each persistent CTA,
// and a slice's tiles go to the CTA's warps in turn.  A warp loads its own tiles
// (four bulk copies of 1152 bytes) into a ring of its own, so no warp waits for another
// until the end of a unit, where the warps' sums are joined in shared memory.  A
// unit cut by a slice's end is joined by whichever of its CTAs comes last.  No
// plan kernel: every CTA sums the unions' lengths itself.
#include <limits.h>

#include "dd_attn.cuh"
#include "dd_kv4.cuh"

namespace dd {

namespace {

constexpr int kMaxRuns = 16;             // units of a slice listed at a time
constexpr int kTileBytes = 4 * kBlk4;    // two blocks of 16 rows: K and V of the first, then of the second
constexpr int kJoinRow = 132;            // floats of a query vector's sums in the joining buffer (128 + padding)
constexpr float kLazy = 8.f;             // a score may exceed the reference by 2^kLazy ...
constexpr float kHead = 6.f;             // ... and weights are held times 2^kHead

// NT tiles of 8 query vectors a warp, two CTAs on an SM.  Up to 4 query vectors (kPack)
// the two parts of P share a tile, one in its columns 0-3, one in 4-7, which halves the
// products with V (whole cache, 8 requests of 128K: 195 -> 179 us).  One tile: eight warps a CTA
// with the queries in registers (128 registers a thread); two: six warps (168), the
// queries in shared memory.
__host__ __device__ constexpr int attn4_warps(int nt) { return nt == 1 ? 8 : 6; }
constexpr int kStages = 2;               // tiles in flight per warp
__host__ __device__ constexpr size_t attn4_smem(int nt) {
  return (size_t)attn4_warps(nt) * (kStages * kTileBytes + 8 * kJoinRow * 4) + (nt > 1 ? (size_t)nt * 8 * 256 : 0);
}

struct Run {           // a unit's place in the sequence of tiles
  int vunit, unit, b, g, q0;       // unit and group of query vectors, request, KV head, first query vector
  int start, end, cnt, len;        // tiles [start, end) of the sequence; chunks; rows (INT_MAX: no kv_len)
  int cta0, cta1;                  // the CTAs that share it
  int ke, ve;
};

struct Attn4Params {
  Attn4Args a;
  int NQ, G, bpc_shift, groups, group_q, vunits;   // vunits = units * groups of group_q query vectors
  float *part_o, *part_ml;
  int32_t *arrive;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the first product of a sum: C is zero without registers for it
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// byte i of codes -> half2
__device__ __forceinline__ uint32_t e2m1_byte(uint32_t w, int i) {
  uint32_t r;
#define DD_E2M1_BYTE(B)                                                            \
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n"            \
      " cvt.rn.f16x2.e2m1x2 %0, " B ";\n}\n"                                       \
      : "=r"(r)                                                                    \
      : "r"(w))
  switch (i) {   // a constant once the loops are unrolled
    case 0: DD_E2M1_BYTE("b0"); break;
    case 1: DD_E2M1_BYTE("b1"); break;
    case 2: DD_E2M1_BYTE("b2"); break;
    default: DD_E2M1_BYTE("b3"); break;
  }
#undef DD_E2M1_BYTE
  return r;
}

// transpose of an 8x8 matrix of 16-bit values held in fragment order
__device__ __forceinline__ uint32_t movm(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
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

// Tiles of a unit: pairs of its union's blocks of 16 rows, those wholly behind the
// end left out (chunk numbers ascend, so block x lies at position 16 x or later),
// at least one, so that a unit without rows is visited too.
struct Lengths {
  int cnt, len, exps;      // chunks, rows (INT_MAX without kv_len), ke | ve << 16
};
__device__ __forceinline__ int unit_tiles(const Attn4Params &p, int vunit, Lengths &r) {
  const Attn4Args &a = p.a;
  const int unit = vunit / p.groups, b = unit / a.Hkv, g = unit - b * a.Hkv;
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
  return max((n + 1) >> 1, 1);
}

__device__ __forceinline__ void fill_run(const Attn4Params &p, Run &r, int vunit, int start, int end,
                                         const Lengths &l) {
  r.vunit = vunit;
  r.unit = vunit / p.groups;
  r.q0 = (vunit - r.unit * p.groups) * p.group_q;
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

// Step's own rows (in shared memory: keys, then values; the query vector too), then
// the division.  The lane holds columns 4 lane .. of the query vector.
__device__ __forceinline__ void finish(const Attn4Params &p, int unit, int qv, Part s, const uint2 *query,
                                       const uint2 *tails, int lane) {
  const Attn4Args &a = p.a;
  if (a.k_tail) {
    const float sl2 = a.softmax_scale * 1.4426950408889634f;
    const uint2 qw = query[lane];
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
      const float m = fmaxf(s.m, x);      // a NaN score leaves m: its weight is NaN
      const float wa = weight_of(s.m, m), wt = weight_of(x, m);
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

// fp16 fragments of a lane's 32 query values, scaled by a power of two, and the factor back.  B fragment of
// step s: values 32 t4 + 4 s + {0,1} and {2,3} of query vector g8.
__device__ __forceinline__ void query_fragments(const uint4 (&w)[4], uint32_t (&f)[16], float &back) {
  const uint32_t v[16] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w,
                          w[2].x, w[2].y, w[2].z, w[2].w, w[3].x, w[3].y, w[3].z, w[3].w};
  uint32_t top = 0;   // largest magnitude, as bits
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, max((v[i] & 0x7FFFu) << 16, v[i] & 0x7FFF0000u));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int e = (int)(top >> 23);
  const int sh = top == 0 || e == 255 ? 0 : min(126, 14 - (e - 127));
  const float mul = pow2i(sh);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = cvt_f16x2(bf_lo(v[i]) * mul, bf_hi(v[i]) * mul);
  back = pow2i(-sh);
}

template <int NT, bool kPack>
__global__ void __launch_bounds__(attn4_warps(NT) * 32, 2) k_attn4(const __grid_constant__ Attn4Params p) {
  constexpr int S = kStages, kWarps = attn4_warps(NT), kThreads = kWarps * 32;
  constexpr bool kQReg = NT == 1;
  extern __shared__ __align__(128) uint8_t smem[];
  float *join = reinterpret_cast<float *>(smem + kWarps * S * kTileBytes);     // [kWarps][8][kJoinRow]
  uint8_t *qsm = smem + kWarps * S * kTileBytes + kWarps * 8 * kJoinRow * 4;   // [NT][8 steps][32 lanes][8 B]
  __shared__ __align__(8) uint64_t bars[kWarps * S];
  __shared__ Run runs[kMaxRuns];
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  __shared__ uint4 s_tails[2 * kMaxNq * 16];      // the unit's own new rows: keys, values
  __shared__ float s_back[NT * 8];
  __shared__ int scratch[33];
  __shared__ int s_first, s_flag, s_lo, s_hi;
  __shared__ uint4 s_query[NT * 8 * 16];            // the run's query vectors as they are

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t4 = lane & 3, g8 = lane >> 2;
  const Attn4Args &a = p.a;
  const uint32_t bar0 = smem_u32(bars) + warp * S * 8;
  const uint32_t ring = smem_u32(smem) + warp * S * kTileBytes;
  if (lane < S) mbar_init(bar0 + 8 * lane, 2);   // the two lanes that ask for a tile's blocks
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  pdl_wait();
  pdl_trigger();

  // ------------------------------------------------------------- the slice
  // Equal slices of the sequence, in whole rounds of the warps.  A slice that holds the
  // end of one unit and the start of the next pays for two queries and two joins, two
  // to three rounds' time, so where the units are no more than the threads (their
  // lengths are then loaded once) and parts of up to two rounds more than a slice let
  // every CTA work on one unit, the units are cut into such parts instead.
  // Llama-3-8B layer, two queries: 21.0 -> 18.8 us; three requests, 21 units: 32.4 -> 20.8 us.
  const bool one_round = p.vunits <= kThreads;
  if (tid == 0) s_flag = load_status(a.status);
  const int64_t staged = a.miss_count ? min((int64_t)*a.miss_count, a.max_misses) : a.max_misses;
  Lengths mine{};
  int my_tiles = 0, my_start, total;
  if (one_round) {
    if (tid < p.vunits) my_tiles = unit_tiles(p, tid, mine);
    my_start = block_excl_scan(my_tiles, scratch, &total);
  } else {
    for (int u = tid; u < p.vunits; u += kThreads) my_tiles += unit_tiles(p, u, mine);
    total = block_sum(my_tiles, scratch);
  }
  const bool dead = s_flag != 0;       // an error is pending: no work (the counts below still go on)
  const int n_cta = (int)gridDim.x;
  int per = ((total + n_cta - 1) / n_cta + kWarps - 1) / kWarps * kWarps;
  int lo = (int)min((int64_t)total, (int64_t)blockIdx.x * per), hi = min(total, lo + per);
  bool parts = false;
  if (one_round && n_cta + kThreads < 1024) {
    // the number of parts for three part lengths, 10 bits each (at most n_cta + units)
    int mine3 = 0, all3;
#pragma unroll
    for (int k = 0; k < 3; ++k) mine3 |= (my_tiles + per + k * kWarps - 1) / (per + k * kWarps) << (10 * k);
    const int before3 = block_excl_scan(mine3, scratch, &all3);
#pragma unroll
    for (int k = 2; k >= 0; --k) {
      if ((all3 >> (10 * k) & 1023) > n_cta) continue;
      parts = true;
      const int n = mine3 >> (10 * k) & 1023, first = before3 >> (10 * k) & 1023;
      const int part = (int)blockIdx.x - first;
      if (k == 0 || (all3 >> (10 * (k - 1)) & 1023) > n_cta) {      // the shortest that fits
        hi = (int)blockIdx.x < (all3 >> (10 * k) & 1023);           // does this CTA have a part?
        lo = 0;
        if (n && part >= 0 && part < n) {
          const int len = (my_tiles + n - 1) / n;
          fill_run(p, runs[0], tid, my_start, my_start + my_tiles, mine);
          runs[0].cta0 = first;
          runs[0].cta1 = first + n - 1;
          s_lo = my_start + part * len;
          s_hi = min(my_start + my_tiles, s_lo + len);
        }
        break;
      }
    }
  }
  if (lo >= hi) return;
  const int64_t page = (int64_t)16 * kRow4 << p.bpc_shift;
  const uint32_t all_q = (1u << a.n_q) - 1u;
  const float sl2 = a.softmax_scale * 1.4426950408889634f;

  uint32_t seq = 0;                    // tiles this warp has been through: stage and phase
  bool alive = true;

  for (int w0 = 0;; w0 += kMaxRuns) {
    // the slice's units number w0 .. w0 + kMaxRuns - 1; the barrier is for what this list
    // and s_lo, s_hi held before, and for the part written above
    __syncthreads();
    int n_seen = 0;                    // units of the slice seen
    if (parts) {
      n_seen = 1;
      lo = s_lo;
      hi = s_hi;
    } else {
      int base = 0;                    // tiles of the units before this round
      for (int u0 = 0; u0 < p.vunits && base < hi; u0 += kThreads) {
        int all = total, start = my_start;
        if (!one_round) {
          const int u = u0 + tid;
          my_tiles = u < p.vunits ? unit_tiles(p, u, mine) : 0;
          start = base + block_excl_scan(my_tiles, scratch, &all);
        }
        const bool in = my_tiles && start < hi && start + my_tiles > lo;
        if (in && start <= lo) s_first = u0 + tid;
        const int n = __syncthreads_count(in);
        if (n) {
          const int rank = u0 + tid - s_first - w0;
          if (in && rank >= 0 && rank < kMaxRuns) {
            fill_run(p, runs[rank], u0 + tid, start, start + my_tiles, mine);
            runs[rank].cta0 = start / per;
            runs[rank].cta1 = (start + my_tiles - 1) / per;
          }
          n_seen += n;
        }
        base += all;
      }
      __syncthreads();
    }
    const int n_runs = min(n_seen - w0, kMaxRuns);
    const int wlo = max(lo, runs[0].start), whi = min(hi, runs[n_runs - 1].end);

    // --------------------------------------- this warp's tiles: wlo + warp + i * kWarps
    const int n_tiles = whi - wlo > warp ? (whi - wlo - warp + kWarps - 1) / kWarps : 0;
    // the first run's query vectors are on their way while the tiles are looked up
    // a run's query vectors and its own new rows come by asynchronous copies, the first
    // run's while its tiles are looked up
    auto stage_run = [&](const Run &r) {
      for (int e = tid; e < NT * 8 * 16; e += kThreads) {
        const int qv = r.q0 + (e >> 4);
        if (qv < p.NQ)
          cp_async16(s_query + e, reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + out_row(p, r.unit, qv)) + (e & 15));
        else
          s_query[e] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (a.k_tail) {
        for (int i = tid; i < 2 * a.n_q * 16; i += kThreads) {
          const int kv = i >= a.n_q * 16, e = kv ? i - a.n_q * 16 : i;
          const uint16_t *src = static_cast<const uint16_t *>(kv ? a.v_tail : a.k_tail);
          cp_async16(s_tails + kv * kMaxNq * 16 + e, reinterpret_cast<const uint4 *>(
              src + ((int64_t)(r.b * a.n_q + (e >> 4)) * a.Hkv + r.g) * kD) + (e & 15));
        }
      }
    };
    stage_run(runs[0]);
    // lane 2 t + h holds block h of tile i0 + t: its slot, and {query mask, rows in use << 8, block of the chunk << 13}
    auto entry = [&](int i, int &slot, uint32_t &meta) {
      slot = 0;
      meta = 0;
      if (i >= n_tiles || dead) return;
      const int x = wlo + warp + i * kWarps;
      int r = 0;
#pragma unroll
      for (int step = kMaxRuns / 2; step > 0; step >>= 1)
        if (r + step < n_runs && runs[r + step].start <= x) r += step;
      const int blk = 2 * (x - runs[r].start) + (lane & 1);
      const int ci = blk >> p.bpc_shift, sub = blk & ((1 << p.bpc_shift) - 1);
      if (ci >= runs[r].cnt) return;
      const int64_t e = (int64_t)runs[r].unit * a.umax + ci;
      slot = a.union_slot[e];
      const uint32_t qm = a.union_qmask ? a.union_qmask[e] & all_q : all_q;
      int rows = 16;
      if (a.kv_len) {
        const int64_t left = runs[r].len - ((int64_t)a.union_idx[e] * a.cs + sub * 16);
        rows = left < 0 ? 0 : left > 16 ? 16 : (int)left;
      }
      if (slot >= 0 ? slot >= a.hot_slots : -1 - (int64_t)slot >= staged) {
        set_status(a.status, DD_ERR_DEVICE_CHECK);
        rows = 0;
      }
      if (qm && rows) meta = qm | (uint32_t)rows << 8 | (uint32_t)sub << 13;
    };
    int cur_slot, nxt_slot = 0, i0 = 0;
    uint32_t cur_meta, nxt_meta = 0;
    entry(lane >> 1, cur_slot, cur_meta);

    // the two lanes that hold tile i ask for its blocks (an empty block just arrives)
    auto issue = [&](int i) {
      if (i < n_tiles && (lane >> 1) == (i & 15)) {
        const bool n = i >= i0 + 16;
        const int slot = n ? nxt_slot : cur_slot;
        const uint32_t meta = n ? nxt_meta : cur_meta;
        const uint32_t st = (seq + (uint32_t)i) % S, bar = bar0 + 8 * st;
        if (meta && alive) {
          const int64_t off = (slot >= 0 ? (int64_t)slot : -1 - (int64_t)slot) * page + (int64_t)(meta >> 13) * kBlk4;
          const uint32_t dst = ring + st * kTileBytes + (lane & 1) * 2 * kBlk4;
          mbar_arrive_expect_tx(bar, 2 * kBlk4);
          bulk_load(dst, (slot >= 0 ? a.Khot : a.Kst) + off, kBlk4, bar);
          bulk_load(dst + kBlk4, (slot >= 0 ? a.Vhot : a.Vst) + off, kBlk4, bar);
        } else {
          mbar_arrive(bar);
        }
      }
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) issue(i);
    entry(16 + (lane >> 1), nxt_slot, nxt_meta);

    int i = 0;
#pragma unroll 1
    for (int r = 0; r < n_runs; ++r) {
      const int unit = runs[r].unit, q0 = runs[r].q0, run_end = runs[r].end;
      const float kmul = sl2 * pow2i(runs[r].ke);
      uint32_t qf[16];            // one tile: its fragments
      float mul[NT][2];           // score units of columns 2 t4 and 2 t4 + 1
      int jq[NT][2];              // their queries (31: no such query vector)
      cp_async_wait_all();
      __syncthreads();
      if constexpr (kQReg) {
        uint4 w[4];
        float back;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = s_query[(kPack ? g8 & 3 : g8) * 16 + t4 * 4 + e];
        query_fragments(w, qf, back);
        mul[0][0] = __shfl_sync(0xffffffffu, back, t4 * 8) * kmul;
        mul[0][1] = __shfl_sync(0xffffffffu, back, t4 * 8 + 4) * kmul;
      } else {
        if (warp < NT) {
          uint4 w[4];
          uint32_t f[16];
          float back;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = s_query[(warp * 8 + g8) * 16 + t4 * 4 + e];
          query_fragments(w, f, back);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            *reinterpret_cast<uint2 *>(qsm + ((warp * 8 + s) * 32 + lane) * 8) = make_uint2(f[2 * s], f[2 * s + 1]);
          if (t4 == 0) s_back[warp * 8 + g8] = back;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mul[n][0] = s_back[n * 8 + 2 * t4] * kmul;
          mul[n][1] = s_back[n * 8 + 2 * t4 + 1] * kmul;
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int qv = q0 + n * 8 + (kPack ? (2 * t4 + c) & 3 : 2 * t4 + c);
          jq[n][c] = qv < p.NQ ? qv / p.G : 31;
        }

      float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[n][e][0] = o[n][e][1] = o[n][e][2] = o[n][e][3] = 0.f;
      }

#pragma unroll 1
      for (; i < n_tiles && wlo + warp + i * kWarps < run_end; ++i) {
        // a block that was not asked for (0) is computed with all its rows masked
        const uint32_t meta0 = __shfl_sync(0xffffffffu, cur_meta, 2 * (i & 15));
        const uint32_t meta1 = __shfl_sync(0xffffffffu, cur_meta, 2 * (i & 15) + 1);
        const uint32_t st = (seq + (uint32_t)i) % S;
        if (!mbar_wait(bar0 + 8 * st, ((seq + (uint32_t)i) / S) & 1, a.status)) alive = false;
        alive = __all_sync(0xffffffffu, alive);
        if ((meta0 | meta1) && alive) {
          const uint32_t tile = ring + st * kTileBytes;
          const uint32_t full_meta = all_q | 16u << 8;
          const bool full = (meta0 & 0x1FFFu) == full_meta && (meta1 & 0x1FFFu) == full_meta;
          // row r of an A fragment is row r ^ (r >> 1 & 1) of each half block: the four
          // V rows that a quarter of a warp loads then spread over both halves of the banks
          const int kr = g8 ^ (g8 >> 1 & 1);

          // ---- S^T = K Q^T
          float c[2][NT][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t kb = tile + h * 2 * kBlk4;
            const uint4 w0 = lds128(kb + kr * 64 + t4 * 16), w1 = lds128(kb + (kr + 8) * 64 + t4 * 16);
            const uint32_t s0 = e4m3x2_to_half2(lds16(kb + kBlk4Scales + kr * 8 + t4 * 2));
            const uint32_t s1 = e4m3x2_to_half2(lds16(kb + kBlk4Scales + (kr + 8) * 8 + t4 * 2));
            const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w}, wb[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t sa = __byte_perm(s0, 0u, w < 2 ? 0x1010 : 0x3232);
              const uint32_t sb = __byte_perm(s1, 0u, w < 2 ? 0x1010 : 0x3232);
              uint32_t ha[4], hb[4];
              e2m1x8_to_half2(wa[w], ha);
              e2m1x8_to_half2(wb[w], hb);
#pragma unroll
              for (int e = 0; e < 4; ++e) ha[e] = hmul2_u32(ha[e], sa), hb[e] = hmul2_u32(hb[e], sb);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t af[4] = {ha[2 * e], hb[2 * e], ha[2 * e + 1], hb[2 * e + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  uint2 q2;
                  if constexpr (kQReg)
                    q2 = make_uint2(qf[2 * (2 * w + e)], qf[2 * (2 * w + e) + 1]);
                  else
                    q2 = *reinterpret_cast<const uint2 *>(qsm + ((n * 8 + 2 * w + e) * 32 + lane) * 8);
                  if (w == 0 && e == 0)
                    mma_f16_first(c[h][n], af, q2.x, q2.y);
                  else
                    mma_f16(c[h][n], af, q2.x, q2.y);
                }
              }
            }
          }

          // ---- softmax, and P^T as two fp16 parts
          uint32_t ph[2][NT][2], pl[2][NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[h][e] = c[h][n][e] * mul[n][e & 1];
            if (!full) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t meta = h ? meta1 : meta0;
                const int rows = (int)(meta >> 8) & 31;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!((meta & 255u) >> jq[n][e & 1] & 1u) || kr + (e >> 1) * 8 >= rows) x[h][e] = -INFINITY;
              }
            }
            float t0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
            float t1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
            if (__any_sync(0xffffffffu, t0 > m[n][0] + (kLazy + kHead) || t1 > m[n][1] + (kLazy + kHead))) {
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
              }
              const float n0 = fmaxf(m[n][0], t0 - kHead), n1 = fmaxf(m[n][1], t1 - kHead);
              const float a0 = weight_of(m[n][0], n0), a1 = weight_of(m[n][1], n1);
              m[n][0] = n0;
              m[n][1] = n1;
              l[n][0] *= a0;
              l[n][1] *= a1;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                o[n][e][0] *= a0;
                o[n][e][1] *= a1;
                o[n][e][2] *= a0;
                o[n][e][3] *= a1;
              }
            }
            // a column without a row so far: -inf - 0 gives weight 0, and a NaN passes
            const float b0 = m[n][0] == -INFINITY ? 0.f : m[n][0], b1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float p0 = ex2_approx(x[h][0] - b0), p1 = ex2_approx(x[h][1] - b1);
              const float p2 = ex2_approx(x[h][2] - b0), p3 = ex2_approx(x[h][3] - b1);
              l[n][0] += p0 + p2;
              l[n][1] += p1 + p3;
              const uint32_t h0 = cvt_f16x2(p0, p1), h1 = cvt_f16x2(p2, p3);
              const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
              const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
              const uint32_t l0 = cvt_f16x2(p0 - f0.x, p1 - f0.y), l1 = cvt_f16x2(p2 - f1.x, p3 - f1.y);
              if constexpr (kPack) {   // columns 0-3: the first part, 4-7: the second
                ph[h][n][0] = movm(t4 < 2 ? h0 : l0);
                ph[h][n][1] = movm(t4 < 2 ? h1 : l1);
              } else {
                ph[h][n][0] = movm(h0);
                ph[h][n][1] = movm(h1);
                pl[h][n][0] = movm(l0);
                pl[h][n][1] = movm(l1);
              }
            }
          }

          // ---- O^T += V^T P^T: rows k = 2 t4, 2 t4 + 1 and 8 more of each block, columns 16 g8 ..
          {
            const int ra = 2 * t4 ^ (t4 & 1), rb = ra ^ 1;
            uint32_t sc[2], bad_rows = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t vs = tile + (2 * h + 1) * kBlk4 + kBlk4Scales + g8;
              sc[h] = lds8(vs + ra * 8) | lds8(vs + rb * 8) << 8 | lds8(vs + (ra + 8) * 8) << 16 |
                      lds8(vs + (rb + 8) * 8) << 24;
              if (!full) {   // rows behind the end may hold anything: scale 0
                const int rows = (int)((h ? meta1 : meta0) >> 8) & 31;
                if (ra >= rows) sc[h] &= 0xFFFFFF00u;
                if (rb >= rows) sc[h] &= 0xFFFF00FFu;
                if (ra + 8 >= rows) sc[h] &= 0xFF00FFFFu;
                if (rb + 8 >= rows) sc[h] &= 0x00FFFFFFu;
              }
              bad_rows |= (sc[h] & 0x7F7F7F7Fu) + 0x01010101u;
            }
            if (__any_sync(0xffffffffu, (bad_rows & 0x80808080u) != 0u)) {
              // a NaN group of V: its columns become NaN for the queries that see the block, and it is
              // left out of the products, where 0 * NaN would reach every query
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t nan = ((sc[h] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                sc[h] &= ~((nan >> 7) * 0xFFu);
                const unsigned bad = __ballot_sync(0xffffffffu, nan != 0u);
                const bool mine = (bad >> (lane & 28)) & 15u;     // any of the block's rows, columns 16 g8 ..
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (mine && (((h ? meta1 : meta0) & 255u) >> jq[n][e & 1] & 1u)) {
#pragma unroll
                      for (int t = 0; t < 8; ++t) o[n][t][e] = NAN;
                    }
              }
            }
            const uint32_t s01[2] = {e4m3x2_to_half2(sc[0]), e4m3x2_to_half2(sc[1])};
            const uint32_t s23[2] = {e4m3x2_to_half2(sc[0] >> 16), e4m3x2_to_half2(sc[1] >> 16)};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              // even columns of two rows side by side, then the odd ones
              uint32_t x[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t vb = tile + (2 * h + 1) * kBlk4 + g8 * 8 + 4 * w + e * 512;
                  const uint32_t xa = lds32(vb + ra * 64), xb = lds32(vb + rb * 64);
                  x[h][2 * e] = (xa & 0x0F0F0F0Fu) | ((xb << 4) & 0xF0F0F0F0u);
                  x[h][2 * e + 1] = ((xa >> 4) & 0x0F0F0F0Fu) | (xb & 0xF0F0F0F0u);
                }
#pragma unroll
              for (int t2 = 0; t2 < 4; t2 += 2) {
                uint32_t af[2][2][4];
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      af[q][h][e] = hmul2_u32(e2m1_byte(x[h][e], t2 + q), e < 2 ? s01[h] : s23[h]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  float d[2][4];
                  // two sums at a time: a product waits for the one before it in its sum
#pragma unroll
                  for (int q = 0; q < 2; ++q) mma_f16_first(d[q], af[q][0], ph[0][n][0], ph[0][n][1]);
#pragma unroll
                  for (int q = 0; q < 2; ++q) mma_f16(d[q], af[q][1], ph[1][n][0], ph[1][n][1]);
                  if constexpr (!kPack) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) mma_f16(d[q], af[q][0], pl[0][n][0], pl[0][n][1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) mma_f16(d[q], af[q][1], pl[1][n][0], pl[1][n][1]);
                  }
#pragma unroll
                  for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][4 * w + t2 + q][e] += d[q][e];
                }
              }
            }
          }
        }
        __syncwarp();
        issue(i + S);
        if ((i & 15) == 15) {
          i0 += 16;
          cur_slot = nxt_slot;
          cur_meta = nxt_meta;
          entry(i0 + 16 + (lane >> 1), nxt_slot, nxt_meta);
        }
      }

      // ------------------------------------------------ join the warps, 8 query vectors at a time
      const int vunit = runs[r].vunit;
      const int cta0 = runs[r].cta0, cta1 = runs[r].cta1;
      const bool shared = cta0 != cta1;
      const float vmul = pow2i(runs[r].ve);
      const uint2 *tails = reinterpret_cast<const uint2 *>(s_tails);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float l0 = l[n][0], l1 = l[n][1];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l0 += __shfl_xor_sync(0xffffffffu, l0, d);
          l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        if (g8 == 0) {
          s_m[warp][2 * t4] = m[n][0], s_m[warp][2 * t4 + 1] = m[n][1];
          s_l[warp][2 * t4] = l0, s_l[warp][2 * t4 + 1] = l1;
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          float *dst = join + (warp * 8 + 2 * t4 + cc) * kJoinRow + 16 * g8;
#pragma unroll
          for (int t = 0; t < 4; ++t)
            *reinterpret_cast<float4 *>(dst + 4 * t) = make_float4(o[n][2 * t][cc], o[n][2 * t][2 + cc],
                                                                   o[n][2 * t + 1][cc], o[n][2 * t + 1][2 + cc]);
        }
        __syncthreads();
#pragma unroll 1
        for (int k = warp; k < (kPack ? 4 : 8); k += kWarps) {
          const int qv = q0 + n * 8 + k;        // this warp's query vector
          if (qv >= p.NQ || dead) break;
          Part s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) s.m = fmaxf(s.m, s_m[w][k]);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float wt = weight_of(s_m[w][k], s.m);
            float4 v = *reinterpret_cast<const float4 *>(join + (w * 8 + k) * kJoinRow + 4 * lane);
            if constexpr (kPack) {
              const float4 v2 = *reinterpret_cast<const float4 *>(join + (w * 8 + 4 + k) * kJoinRow + 4 * lane);
              v.x += v2.x, v.y += v2.y, v.z += v2.z, v.w += v2.w;
            }
            s.l = fmaf(wt, s_l[w][k], s.l);
            s.o.x = fmaf(wt, v.x, s.o.x);
            s.o.y = fmaf(wt, v.y, s.o.y);
            s.o.z = fmaf(wt, v.z, s.o.z);
            s.o.w = fmaf(wt, v.w, s.o.w);
          }
          s.o.x *= vmul, s.o.y *= vmul, s.o.z *= vmul, s.o.w *= vmul;
          if (!shared) {
            finish(p, unit, qv, s, reinterpret_cast<const uint2 *>(s_query + (n * 8 + k) * 16), tails, lane);
          } else {
            const int64_t at = ((int64_t)blockIdx.x + vunit) * (NT * 8) + n * 8 + k;
            *reinterpret_cast<float4 *>(p.part_o + at * kD + 4 * lane) = s.o;
            if (lane == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(s.m, s.l);
          }
        }
        __syncthreads();
      }
      if (shared) {
        // the barrier above orders the CTA's parts before the count, the one below the count before the reads
        if (tid == 0) {
          const bool last = atom_add_acq_rel_gpu(p.arrive + vunit, 1) == cta1 - cta0;
          if (last) p.arrive[vunit] = 0;        // for the next call
          s_flag = last;
        }
        __syncthreads();
        const bool last = s_flag != 0;
        if (last && !dead) {
#pragma unroll 1
          for (int k = warp; k < NT * 8; k += kWarps) {
            const int qv = q0 + k;
            if (qv >= p.NQ) break;
            // 32 parts at a time: a lane holds one's reference and weight, the sums of eight are in flight
            Part s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
            for (int k0 = cta0; k0 <= cta1; k0 += 32) {
              const int np = min(32, cta1 - k0 + 1);
              const int64_t at0 = ((int64_t)k0 + vunit) * (NT * 8) + k;
              float2 ml = make_float2(-INFINITY, 0.f);
              if (lane < np) ml = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + 2 * (at0 + (int64_t)lane * (NT * 8))));
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
                float4 v[8];
#pragma unroll
                for (int t = 0; t < 8; ++t)
                  v[t] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + (at0 + (int64_t)min(t0 + t, np - 1) * (NT * 8)) * kD + 4 * lane));
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
            finish(p, unit, qv, s, reinterpret_cast<const uint2 *>(s_query + k * 16), tails, lane);
          }
        }
        __syncthreads();   // s_flag, the tails and the query vectors are read
      }
      if (r + 1 < n_runs) stage_run(runs[r + 1]);
    }
    seq += (uint32_t)n_tiles;
    if (whi >= hi) return;
  }
}

// Up to 8 query vectors: one tile a warp; more: groups of up to 16, each of which goes
// through the unit's pages by itself.
void attn4_tiles(int NQ, int &nt, int &groups) {
  nt = NQ <= 8 ? 1 : 2;
  groups = (NQ + nt * 8 - 1) / (nt * 8);
}

template <int NT, bool kPack>
cudaError_t launch_t(int grid, const Attn4Params &p, cudaStream_t s) {
  cudaError_t e = set_dyn_smem((const void *)k_attn4<NT, kPack>, attn4_smem(NT));
  if (e != cudaSuccess) return e;
  return launch_k(k_attn4<NT, kPack>, dim3(grid), dim3(attn4_warps(NT) * 32), attn4_smem(NT), s, p);
}

}  // namespace

Attn4Plan attn4_plan(int units, int NQ, int sm_count) {
  Attn4Plan pl;
  attn4_tiles(NQ, pl.nt, pl.groups);
  pl.n_cta = sm_count > 0 ? sm_count * 2 : 1;
  const int64_t slots = (int64_t)pl.n_cta + (int64_t)units * pl.groups;
  pl.part_o_floats = slots * pl.nt * 8 * kD;
  pl.part_ml_floats = slots * pl.nt * 8 * 2;
  return pl;
}

cudaError_t launch_attn4(const Attn4Args &a, const Attn4Plan &pl, float *part_o, float *part_ml, int32_t *arrive,
                         cudaStream_t s) {
  Attn4Params p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.NQ = a.n_q * p.G;
  p.bpc_shift = a.cs == 16 ? 0 : a.cs == 32 ? 1 : 2;
  p.groups = pl.groups;
  p.group_q = pl.nt * 8;
  p.vunits = a.B * a.Hkv * pl.groups;
  p.part_o = part_o, p.part_ml = part_ml, p.arrive = arrive;
  // no more CTAs than slices of a tile per warp there can be
  const int kWarps = attn4_warps(pl.nt);
  const int64_t most = ((int64_t)p.vunits * ((((int64_t)a.umax << p.bpc_shift) + 1) / 2 + 1) + kWarps - 1) / kWarps;
  const int grid = (int)(most < pl.n_cta ? most : pl.n_cta);
  if (pl.nt == 2) return launch_t<2, false>(grid, p, s);
  return p.NQ <= 4 ? launch_t<1, true>(grid, p, s) : launch_t<1, false>(grid, p, s);
}

}  // namespace dd
