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
#include "dd_attn.cuh"
#include "dd_kv4.cuh"

namespace dd {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRuns = 64;             // units of a slice listed at a time
constexpr int kTileBytes = 4 * kBlk4;    // two blocks of 16 rows: K and V of the first, then of the second
constexpr int kJoinRow = 132;            // floats of a query vector's sums in the joining buffer (128 + padding)
constexpr float kLazy = 8.f;             // a score may exceed the reference by 2^kLazy ...
constexpr float kHead = 6.f;             // ... and weights are held times 2^kHead

// NT tiles of 8 query vectors a warp.  One tile: its query registers fit beside the
// sums of two CTAs' warps on an SM; more tiles read the queries from shared memory.
__host__ __device__ constexpr int attn4_ctas_per_sm(int nt) { return nt <= 2 ? 2 : 1; }
__host__ __device__ constexpr int attn4_stages(int nt) { return nt <= 2 ? 2 : 4; }
__host__ __device__ constexpr size_t attn4_smem(int nt) {
  return (size_t)kWarps * attn4_stages(nt) * kTileBytes + (size_t)kWarps * 8 * kJoinRow * 4 +
         (nt > 1 ? (size_t)nt * 8 * 256 : 0);
}

struct Run {           // a unit's place in the sequence of tiles
  int unit, start, end, cnt;
};

struct Attn4Params {
  Attn4Args a;
  int NQ, G, bpc_shift, groups, vunits;   // vunits = units * groups of query vectors
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

// shared-memory loads by address (asm: the ring is written by bulk copies)
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(p));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(p));
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
__device__ __forceinline__ int unit_tiles(const Attn4Params &p, int vunit, int &cnt) {
  const int unit = vunit / p.groups;
  cnt = p.a.union_cnt[unit];
  if (cnt < 0 || cnt > p.a.umax) {
    set_status(p.a.status, DD_ERR_DEVICE_CHECK);
    cnt = cnt < 0 ? 0 : p.a.umax;
  }
  int n = cnt << p.bpc_shift;
  if (p.a.kv_len) {
    const int len = max(p.a.kv_len[unit / p.a.Hkv], 0);
    n = min(n, (len >> 4) + ((len & 15) != 0));
  }
  return max((n + 1) >> 1, 1);
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

// fp16 fragments of NT x 8 query vectors, scaled, and each column's factor back.
// B fragment of step s: values 32 t4 + 4 s + {0,1} and {2,3} of query vector g8.
__device__ __forceinline__ void load_query(const Attn4Params &p, int unit, int qv, int t4, uint32_t (&f)[16],
                                           float &back) {
  uint4 w[4];
  if (qv < p.NQ) {
    const uint4 *src =
        reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.a.q) + out_row(p, unit, qv) + 32 * t4);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = src[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
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

template <int NT>
__global__ void __launch_bounds__(kThreads, attn4_ctas_per_sm(NT)) k_attn4(const __grid_constant__ Attn4Params p) {
  constexpr int S = attn4_stages(NT);
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
  __shared__ int s_first, s_flag;

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
  if (tid == 0) s_flag = load_status(a.status);
  int c0, total;
  {
    int sum = 0;
    for (int u = tid; u < p.vunits; u += kThreads) sum += unit_tiles(p, u, c0);
    total = block_sum(sum, scratch);
  }
  const bool dead = s_flag != 0;       // an error is pending: no work (the counts below still go on)
  const int per = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kWarps);
  const int lo = (int)min((int64_t)total, (int64_t)blockIdx.x * per), hi = min(total, lo + per);
  if (lo >= hi) return;
  const int64_t staged = a.miss_count ? min((int64_t)*a.miss_count, a.max_misses) : a.max_misses;
  const int64_t page = (int64_t)16 * kRow4 << p.bpc_shift;
  const uint32_t all_q = (1u << a.n_q) - 1u;
  const float sl2 = a.softmax_scale * 1.4426950408889634f;

  uint32_t seq = 0;                    // tiles this warp has been through: stage and phase
  bool alive = true;

  for (int w0 = 0;; w0 += kMaxRuns) {
    // the slice's units number w0 .. w0 + kMaxRuns - 1
    __syncthreads();
    int base = 0, n_seen = 0;          // tiles of the units before this round, units of the slice seen
    for (int u0 = 0; u0 < p.vunits && base < hi; u0 += kThreads) {
      int cnt = 0;
      const int u = u0 + tid;
      const int v = u < p.vunits ? unit_tiles(p, u, cnt) : 0;
      int all;
      const int start = base + block_excl_scan(v, scratch, &all);
      if (v && start <= lo && lo < start + v) s_first = u;
      __syncthreads();
      if (base + all > lo) {
        const int rank = u - s_first - w0;
        if (v && start < hi && start + v > lo && rank >= 0 && rank < kMaxRuns)
          runs[rank] = Run{u, start, start + v, cnt};
        n_seen += __syncthreads_count(v && start < hi && start + v > lo);
      }
      base += all;
    }
    const int n_runs = min(n_seen - w0, kMaxRuns);
    const int wlo = max(lo, runs[0].start), whi = min(hi, runs[n_runs - 1].end);

    // --------------------------------------- this warp's tiles: wlo + warp + i * kWarps
    const int n_tiles = whi - wlo > warp ? (whi - wlo - warp + kWarps - 1) / kWarps : 0;
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
      const int unit = runs[r].unit / p.groups;
      const int64_t e = (int64_t)unit * a.umax + ci;
      slot = a.union_slot[e];
      const uint32_t qm = a.union_qmask ? a.union_qmask[e] & all_q : all_q;
      int rows = 16;
      if (a.kv_len) {
        const int64_t left = (int64_t)a.kv_len[unit / a.Hkv] - ((int64_t)a.union_idx[e] * a.cs + sub * 16);
        rows = left < 0 ? 0 : left > 16 ? 16 : (int)left;
      }
      if (slot >= 0 ? slot >= a.hot_slots : -1 - (int64_t)slot >= staged) {
        set_status(a.status, DD_ERR_DEVICE_CHECK);
        rows = 0;
      }
      if (qm && rows) meta = qm | (uint32_t)rows << 8 | (uint32_t)sub << 13;
    };
    int cur_slot, nxt_slot, i0 = 0;
    uint32_t cur_meta, nxt_meta;
    entry(lane >> 1, cur_slot, cur_meta);
    entry(16 + (lane >> 1), nxt_slot, nxt_meta);

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

    int i = 0;
#pragma unroll 1
    for (int r = 0; r < n_runs; ++r) {
      const Run run = runs[r];
      const int unit = run.unit / p.groups, qg0 = (run.unit - unit * p.groups) * NT * 8;
      const int b = unit / a.Hkv, g = unit - b * a.Hkv;
      const float kmul = sl2 * pow2i(head_exp(a.k_exp, g, a.status));
      uint32_t qf[16];            // one tile: its fragments
      float mul[NT][2];           // score units of columns 2 t4 and 2 t4 + 1
      int jq[NT][2];              // their queries (31: no such query vector)
      if (a.k_tail && tid < 2 * a.n_q * 16) {
        const int kv = tid >= a.n_q * 16, e = kv ? tid - a.n_q * 16 : tid;
        const uint16_t *src = static_cast<const uint16_t *>(kv ? a.v_tail : a.k_tail);
        s_tails[kv * kMaxNq * 16 + e] = reinterpret_cast<const uint4 *>(
            src + ((int64_t)(b * a.n_q + (e >> 4)) * a.Hkv + g) * kD)[e & 15];
      }
      if constexpr (kQReg) {
        float back;
        load_query(p, unit, qg0 + g8, t4, qf, back);
        mul[0][0] = __shfl_sync(0xffffffffu, back, t4 * 8) * kmul;
        mul[0][1] = __shfl_sync(0xffffffffu, back, t4 * 8 + 4) * kmul;
      } else {
        if (warp < NT) {
          uint32_t f[16];
          float back;
          load_query(p, unit, qg0 + warp * 8 + g8, t4, f, back);
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
          const int qv = qg0 + n * 8 + 2 * t4 + c;
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
      for (; i < n_tiles && wlo + warp + i * kWarps < run.end; ++i) {
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
              ph[h][n][0] = movm(h0);
              ph[h][n][1] = movm(h1);
              pl[h][n][0] = movm(cvt_f16x2(p0 - f0.x, p1 - f0.y));
              pl[h][n][1] = movm(cvt_f16x2(p2 - f1.x, p3 - f1.y));
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
            uint2 v[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t vb = tile + (2 * h + 1) * kBlk4 + g8 * 8;
              v[h][0] = lds64(vb + ra * 64), v[h][1] = lds64(vb + rb * 64);
              v[h][2] = lds64(vb + (ra + 8) * 64), v[h][3] = lds64(vb + (rb + 8) * 64);
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              // even columns of two rows side by side, then the odd ones
              uint32_t x[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t xa = w ? v[h][2 * e].y : v[h][2 * e].x, xb = w ? v[h][2 * e + 1].y : v[h][2 * e + 1].x;
                  x[h][2 * e] = (xa & 0x0F0F0F0Fu) | ((xb << 4) & 0xF0F0F0F0u);
                  x[h][2 * e + 1] = ((xa >> 4) & 0x0F0F0F0Fu) | (xb & 0xF0F0F0F0u);
                }
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                uint32_t af[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int e = 0; e < 4; ++e) af[h][e] = hmul2_u32(e2m1_byte(x[h][e], t), e < 2 ? s01[h] : s23[h]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  float d[4];
                  mma_f16_first(d, af[0], pl[0][n][0], pl[0][n][1]);
                  mma_f16(d, af[1], pl[1][n][0], pl[1][n][1]);
                  mma_f16(d, af[0], ph[0][n][0], ph[0][n][1]);
                  mma_f16(d, af[1], ph[1][n][0], ph[1][n][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[n][4 * w + t][e] += d[e];
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
      const int cta0 = run.start / per, cta1 = (run.end - 1) / per;
      const bool shared = cta0 != cta1;
      const float vmul = pow2i(head_exp(a.v_exp, g, a.status));
      const uint2 *tails = reinterpret_cast<const uint2 *>(s_tails);
      uint2 qw[NT];                // columns 4 lane .. of this warp's query vectors, for the tails
      if (a.k_tail) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int qv = min(qg0 + n * 8 + warp, p.NQ - 1);
          qw[n] = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + out_row(p, unit, qv) + 4 * lane);
        }
      }
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
        const int qv = qg0 + n * 8 + warp;      // this warp's query vector
        if (qv < p.NQ && !dead) {
          Part s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) s.m = fmaxf(s.m, s_m[w][warp]);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float wt = weight_of(s_m[w][warp], s.m);
            const float4 v = *reinterpret_cast<const float4 *>(join + (w * 8 + warp) * kJoinRow + 4 * lane);
            s.l = fmaf(wt, s_l[w][warp], s.l);
            s.o.x = fmaf(wt, v.x, s.o.x);
            s.o.y = fmaf(wt, v.y, s.o.y);
            s.o.z = fmaf(wt, v.z, s.o.z);
            s.o.w = fmaf(wt, v.w, s.o.w);
          }
          s.o.x *= vmul, s.o.y *= vmul, s.o.z *= vmul, s.o.w *= vmul;
          if (!shared) {
            finish(p, unit, qv, s, qw[n], tails, lane);
          } else {
            const int64_t k = ((int64_t)blockIdx.x + run.unit) * (NT * 8) + n * 8 + warp;
            *reinterpret_cast<float4 *>(p.part_o + k * kD + 4 * lane) = s.o;
            if (lane == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * k) = make_float2(s.m, s.l);
          }
        }
        __syncthreads();
      }
      if (shared) {
        // the barrier above orders the CTA's parts before the count, the one below the count before the reads
        if (tid == 0) {
          const bool last = atom_add_acq_rel_gpu(p.arrive + run.unit, 1) == cta1 - cta0;
          if (last) p.arrive[run.unit] = 0;     // for the next call
          s_flag = last;
        }
        __syncthreads();
        const bool last = s_flag != 0;
        if (last && !dead) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int qv = qg0 + n * 8 + warp;
            if (qv >= p.NQ) break;
            Part s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
            for (int k0 = cta0; k0 <= cta1; k0 += 4) {
              float2 ml[4];
              float4 v[4];
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const int64_t k = ((int64_t)min(k0 + t, cta1) + run.unit) * (NT * 8) + n * 8 + warp;
                ml[t] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + 2 * k));
                v[t] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + k * kD + 4 * lane));
              }
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                if (k0 + t > cta1) break;
                const float mn = fmaxf(s.m, ml[t].x);
                const float wa = weight_of(s.m, mn), wt = weight_of(ml[t].x, mn);
                s.l = s.l * wa + wt * ml[t].y;
                s.o.x = s.o.x * wa + wt * v[t].x;
                s.o.y = s.o.y * wa + wt * v[t].y;
                s.o.z = s.o.z * wa + wt * v[t].z;
                s.o.w = s.o.w * wa + wt * v[t].w;
                s.m = mn;
              }
            }
            finish(p, unit, qv, s, qw[n], tails, lane);
          }
        }
        __syncthreads();   // s_flag is read
      }
    }
    seq += (uint32_t)n_tiles;
    if (whi >= hi) return;
  }
}

// Tiles of 8 query vectors per warp: up to 5 (their sums are 160 registers); more are
// split into two groups, each of which goes through the pages itself.
void attn4_tiles(int NQ, int &nt, int &groups) {
  const int tiles = (NQ + 7) / 8;
  groups = (tiles + 4) / 5;
  nt = (tiles + groups - 1) / groups;
}

template <int NT>
cudaError_t launch_t(int grid, const Attn4Params &p, cudaStream_t s) {
  cudaError_t e = set_dyn_smem((const void *)k_attn4<NT>, attn4_smem(NT));
  if (e != cudaSuccess) return e;
  return launch_k(k_attn4<NT>, dim3(grid), dim3(kThreads), attn4_smem(NT), s, p);
}

}  // namespace

Attn4Plan attn4_plan(int units, int NQ, int sm_count) {
  Attn4Plan pl;
  attn4_tiles(NQ, pl.nt, pl.groups);
  pl.n_cta = sm_count > 0 ? sm_count * attn4_ctas_per_sm(pl.nt) : 1;
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
  p.vunits = a.B * a.Hkv * pl.groups;
  p.part_o = part_o, p.part_ml = part_ml, p.arrive = arrive;
  // no more CTAs than slices of kWarps tiles there can be
  const int64_t most = ((int64_t)p.vunits * ((((int64_t)a.umax << p.bpc_shift) + 1) / 2 + 1) + kWarps - 1) / kWarps;
  const int grid = (int)(most < pl.n_cta ? most : pl.n_cta);
  switch (pl.nt) {
    case 1: return launch_t<1>(grid, p, s);
    case 2: return launch_t<2>(grid, p, s);
    case 3: return launch_t<3>(grid, p, s);
    case 4: return launch_t<4>(grid, p, s);
    case 5: return launch_t<5>(grid, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dd
