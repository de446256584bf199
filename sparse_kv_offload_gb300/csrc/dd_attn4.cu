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
// Whole cache, 8 requests of 128K (842 MB): 177 us on the device in a graph (a call among
// others 182-191), where the copies alone take 131 and everything but the copies 160-176.  A tile of 32 rows takes some 750 instructions: 128 conversions
// and 128 multiplications, 41 to interleave V's rows, 64 additions of sums, the rest loads,
// softmax and moves.
//
// Precision.  A code times its scale is exact in fp16.  A query vector is scaled
// by a power of two to just below 2^15, where its 8-bit significands are exact in
// fp16 down to 2^-32 of its largest value.  P is split into two fp16 parts (22
// bits, next to an exponential of ex2.approx, which is good to 2^-22 itself).  The matrix unit
// truncates when it adds; that is left in for the 128 terms of a score and for 32
// rows of O at a time.  The running sums are added in fp32 outside of it, where
// additions round to nearest: over the hundreds of additions of a long context
// truncation shows (1e-5).
// The softmax's reference value is moved only when a score exceeds it by 2^8, so
// most tiles need no maximum across lanes (P stays at 2^14 or below).
//
// Work split: the unions' tiles of 32 rows (two blocks) of all (request, KV head)
// units, laid end to end, are cut into equal slices, one for each persistent CTA,
// and a slice's tiles go to the CTA's warps in turn.  A warp loads its own tiles
// (four bulk copies of 1152 bytes) into a ring of its own, so no warp waits for another
// until the end of a unit, where the warps' sums are joined in shared memory.  A
// unit cut by a slice's end is joined by whichever of its CTAs comes last.  No
// plan kernel: every CTA sums the unions' lengths itself.
#include "dd_attn4.cuh"

namespace dd {

namespace {

constexpr int kTileBytes = 4 * kBlk4;    // two blocks of 16 rows: K and V of the first, then of the second
constexpr int kJoinRow = 132;            // floats of a query vector's sums in the joining buffer (128 + padding)

// NT tiles of 8 query vectors a warp, two CTAs on an SM.  Up to 4 query vectors (kPack)
// the two parts of P share a tile, one in its columns 0-3, one in 4-7, which halves the
// products with V (whole cache, 8 requests of 128K: 195 -> 179 us), and their queries, a
// kilobyte, wait in shared memory, without which registers spill (179 -> 177; 64 requests of
// 128 chunks 47 -> 45).  One tile: eight warps a CTA (128 registers a thread), two: six (168),
// the queries in shared memory too.
__host__ __device__ constexpr int attn4_warps(int nt) { return nt == 1 ? 8 : 6; }
constexpr int kStages = 2;               // tiles in flight per warp
__host__ __device__ constexpr size_t attn4_smem(int nt) {
  return (size_t)attn4_warps(nt) * (kStages * kTileBytes + 8 * kJoinRow * 4) + (nt > 1 ? (size_t)nt * 8 * 256 : 0);
}

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

template <int NT, bool kPack>
__global__ void __launch_bounds__(attn4_warps(NT) * 32, 2) k_attn4(const __grid_constant__ Attn4Params p) {
  constexpr int S = kStages, kWarps = attn4_warps(NT), kThreads = kWarps * 32;
  constexpr bool kQReg = NT == 1 && !kPack;
  constexpr int kVecs = kPack ? 4 : NT * 8;        // query vectors
  extern __shared__ __align__(128) uint8_t smem[];
  float *join = reinterpret_cast<float *>(smem + kWarps * S * kTileBytes);     // [kWarps][8][kJoinRow]
  uint8_t *qsm = smem + kWarps * S * kTileBytes + kWarps * 8 * kJoinRow * 4;   // [NT][8 steps][32 lanes][8 B]
  __shared__ __align__(8) uint64_t bars[kWarps * S];
  __shared__ PlanSmem plan;
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  __shared__ uint4 s_tails[2 * kMaxNq * 16];      // the unit's own new rows: keys, values
  __shared__ float s_back[NT * 8];
  __shared__ int s_flag;
  __shared__ uint4 s_query[kVecs * 16];             // the run's query vectors as they are
  __shared__ uint2 s_pack[kPack ? 8 * 16 : 1];      // their fragments, [8 steps][query vector, quarter]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t4 = lane & 3, g8 = lane >> 2;
  const Attn4Args &a = p.a;
  const uint32_t bar0 = smem_u32(bars) + warp * S * 8;
  const uint32_t ring = smem_u32(smem) + warp * S * kTileBytes;
  if (lane < S) mbar_init(bar0 + 8 * lane, 2);   // the two lanes that ask for a tile's blocks
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  pdl_wait();
  pdl_trigger();

  Slice<kThreads, kWarps, 1> slice;
  if (!slice.open(p, plan)) return;
  const bool dead = slice.dead;
  const uint32_t all_q = (1u << a.n_q) - 1u;
  const float sl2 = a.softmax_scale * 1.4426950408889634f;
  uint32_t seq = 0;                    // tiles this warp has been through: stage and phase
  bool alive = true;

  for (int w0 = 0;; w0 += kMaxRuns) {
    int wlo, whi;
    const int n_runs = slice.list(p, plan, w0, wlo, whi);
    const Run *runs = plan.runs;

    // --------------------------------------- this warp's tiles: wlo + warp + i * kWarps
    const int n_tiles = whi - wlo > warp ? (whi - wlo - warp + kWarps - 1) / kWarps : 0;
    // a run's query vectors and its own new rows come by asynchronous copies, the first
    // run's while its tiles are looked up
    auto stage_run = [&](const Run &r) {
      for (int e = tid; e < kVecs * 16; e += kThreads) {
        const int qv = e >> 4;
        if (qv < p.NQ)
          cp_async16(s_query + e, reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + out_row(p, r.unit, qv)) + (e & 15));
        else
          s_query[e] = make_uint4(0u, 0u, 0u, 0u);
      }
      stage_tails(p, r, s_tails, tid, kThreads);
    };
    // lane 2 t + h holds block h of tile i0 + t
    auto entry = [&](int i) -> Entry {
      if (i >= n_tiles || dead) return {0, 0, -1, 0, 0u};
      const int x = wlo + warp + i * kWarps;
      int r = 0;
#pragma unroll
      for (int step = kMaxRuns / 2; step > 0; step >>= 1)
        if (r + step < n_runs && runs[r + step].start <= x) r += step;
      return load_entry(p, runs[r], 2 * (x - runs[r].start) + (lane & 1), all_q);
    };
    int i0 = 0;
    const Entry first = entry(lane >> 1);
    stage_run(runs[0]);      // on the way together with the union's entries
    BlockRef cur = look_at(p, first, slice.staged, all_q), nxt = {0, 0u};

    // the two lanes that hold tile i ask for its blocks (an empty block just arrives); nobody
    // does once a wait has run out, as nobody waits then
    auto issue = [&](int i) {
      if (i < n_tiles && (lane >> 1) == (i & 15) && alive) {
        const BlockRef r = i >= i0 + 16 ? nxt : cur;
        const uint32_t st = (seq + (uint32_t)i) % S, bar = bar0 + 8 * st;
        if (r.meta)
          load_block(p, r, ring + st * kTileBytes + (lane & 1) * 2 * kBlk4, bar);
        else
          mbar_arrive(bar);
      }
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) issue(i);
    nxt = look_at(p, entry(16 + (lane >> 1)), slice.staged, all_q);

    int i = 0;
#pragma unroll 1
    for (int r = 0; r < n_runs; ++r) {
      const int unit = runs[r].unit, run_end = runs[r].end;
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
        for (int e = 0; e < 4; ++e) w[e] = s_query[g8 * 16 + t4 * 4 + e];
        // B fragment of step s: values 32 t4 + 4 s + {0,1} and {2,3} of query vector g8
        query_fragments(w, qf, back);
        mul[0][0] = score_factor(__shfl_sync(0xffffffffu, back, t4 * 8), kmul);
        mul[0][1] = score_factor(__shfl_sync(0xffffffffu, back, t4 * 8 + 4), kmul);
      } else {
        if (warp < NT && (!kPack || lane < 16)) {
          uint4 w[4];
          uint32_t f[16];
          float back;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = s_query[(warp * 8 + g8) * 16 + t4 * 4 + e];
          query_fragments(w, f, back, kPack ? 0xFFFFu : 0xFFFFFFFFu);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if constexpr (kPack)
              s_pack[s * 16 + lane] = make_uint2(f[2 * s], f[2 * s + 1]);
            else
              *reinterpret_cast<uint2 *>(qsm + ((warp * 8 + s) * 32 + lane) * 8) = make_uint2(f[2 * s], f[2 * s + 1]);
          if (t4 == 0) s_back[warp * 8 + g8] = back;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int qv = n * 8 + (kPack ? 2 * t4 & 3 : 2 * t4);
          mul[n][0] = score_factor(s_back[qv], kmul);
          mul[n][1] = score_factor(s_back[qv + 1], kmul);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int qv = n * 8 + (kPack ? (2 * t4 + c) & 3 : 2 * t4 + c);
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
      for (; alive && i < n_tiles && wlo + warp + i * kWarps < run_end; ++i) {
        // a block that was not asked for (0) is computed with all its rows masked
        const uint32_t meta0 = __shfl_sync(0xffffffffu, cur.meta, 2 * (i & 15));
        const uint32_t meta1 = __shfl_sync(0xffffffffu, cur.meta, 2 * (i & 15) + 1);
        const uint32_t st = (seq + (uint32_t)i) % S;
        alive = ring_wait<S>(bar0, seq + (uint32_t)i, seq + (uint32_t)min(i + S, n_tiles) - 1u, lane, a.status);
        if (!alive) break;
        if (meta0 | meta1) {
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
                  else if constexpr (kPack)
                    q2 = s_pack[(2 * w + e) * 16 + (lane & 15)];
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
            if (__any_sync(0xffffffffu, t0 > highest_for(m[n][0]) || t1 > highest_for(m[n][1]))) {
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
            uint2 va[2][2], vb[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t at = tile + (2 * h + 1) * kBlk4 + g8 * 8 + e * 512;
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(va[h][e].x), "=r"(va[h][e].y) : "r"(at + ra * 64));
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(vb[h][e].x), "=r"(vb[h][e].y) : "r"(at + rb * 64));
              }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              // even columns of two rows side by side, then the odd ones
              uint32_t x[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t xa = w ? va[h][e].y : va[h][e].x, xb = w ? vb[h][e].y : vb[h][e].x;
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
          cur = nxt;
          nxt = look_at(p, entry(i0 + 16 + (lane >> 1)), slice.staged, all_q);
        }
      }

      // ------------------------------------------------ join the warps, 8 query vectors at a time
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
          const int qv = n * 8 + k;        // this warp's query vector
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
            finish(p, unit, qv, s, reinterpret_cast<const uint2 *>(s_query + (n * 8 + k) * 16)[lane], tails, lane);
          } else {
            const int64_t at = ((int64_t)blockIdx.x + unit) * (NT * 8) + n * 8 + k;
            *reinterpret_cast<float4 *>(p.part_o + at * kD + 4 * lane) = s.o;
            if (lane == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(s.m, s.l);
          }
        }
        __syncthreads();
      }
      if (shared) {
        // the barrier above orders the CTA's parts before the count, the one below the count before the reads
        if (tid == 0) s_flag = arrive_at_unit(p, runs[r], dead);
        __syncthreads();
        if (s_flag) {
#pragma unroll 1
          for (int k = warp; k < p.NQ; k += kWarps)
            finish(p, unit, k, combine_parts(p, runs[r], k, lane),
                   reinterpret_cast<const uint2 *>(s_query + k * 16)[lane], tails, lane);
        }
        __syncthreads();   // s_flag, the tails and the query vectors are read
      }
      if (r + 1 < n_runs) stage_run(runs[r + 1]);
    }
    seq += (uint32_t)n_tiles;
    if (whi >= slice.hi) return;
  }
}

template <int NT, bool kPack>
cudaError_t launch_t(int grid, const Attn4Params &p, cudaStream_t s) {
  cudaError_t e = set_dyn_smem((const void *)k_attn4<NT, kPack>, attn4_smem(NT));
  if (e != cudaSuccess) return e;
  return launch_k(k_attn4<NT, kPack>, dim3(grid), dim3(attn4_warps(NT) * 32), attn4_smem(NT), s, p);
}

}  // namespace

// Up to 8 query vectors: one tile a warp, up to 16: two; more: tcgen05.  Both sides of the
// second border (us on the device, mma.sync in groups of 16 / tcgen05):
//    4  one request, 16 chunks of 16                          6.6 / 10.0
//    4  8 requests of 128K, whole cache, 8 KV heads           177 / 463
//    8  16 requests, 64 of 2,048 chunks of 16, two queries    19.1 / 28.9
//   12  8 requests, 256 of 512 chunks of 64, two queries      41.5 / 63.2
//   15  3 requests, 77 of 333 chunks of 32, three queries     20.9 / 22.0
//   16  32 requests, 128 of 2,048 chunks of 16, four queries  79 / 111
//   20  16 requests, 100 of 512 chunks of 32, two queries     44.3 / 40.9
//   24  2 requests, 64 of 1,024 chunks of 16, two queries     17.5 / 17.3
//   40  32 requests, 128 of 2,048 chunks of 16, five queries  215 / 133
//   64  8 requests, 64 of 1,024 chunks of 32, eight queries   87 / 60
// (The first border is a tile's width: up to it a second tile would hold padding only.)
Attn4Plan attn4_plan(int units, int NQ, int sm_count) {
  Attn4Plan pl;
  pl.nt = NQ <= 8 ? 1 : NQ <= 16 ? 2 : 0;
  pl.group_q = pl.nt ? pl.nt * 8 : (NQ + 7) / 8 * 8;
  pl.n_cta = sm_count > 0 ? sm_count * (pl.nt ? 2 : 1) : 1;
  const int64_t slots = (int64_t)pl.n_cta + units;
  pl.part_o_floats = slots * pl.group_q * kD;
  pl.part_ml_floats = slots * pl.group_q * 2;
  return pl;
}

cudaError_t launch_attn4(const Attn4Args &a, const Attn4Plan &pl, float *part_o, float *part_ml, int32_t *arrive,
                         cudaStream_t s) {
  Attn4Params p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.NQ = a.n_q * p.G;
  p.bpc_shift = a.cs == 16 ? 0 : a.cs == 32 ? 1 : 2;
  p.group_q = pl.group_q;
  p.units = a.B * a.Hkv;
  p.part_o = part_o, p.part_ml = part_ml, p.arrive = arrive;
  // no more CTAs than slices of a tile per warp (tcgen05: of a tile) there can be
  const int tile_blocks = pl.nt ? 2 : 8, quantum = pl.nt ? attn4_warps(pl.nt) : 1;
  const int64_t blocks = (int64_t)a.umax << p.bpc_shift;
  const int64_t most = ((int64_t)p.units * ((blocks + tile_blocks - 1) / tile_blocks + 1) + quantum - 1) / quantum;
  const int grid = (int)(most < pl.n_cta ? most : pl.n_cta);
  if (pl.nt == 0) return launch_attn4_tc(grid, p, s);
  if (pl.nt == 2) return launch_t<2, false>(grid, p, s);
  return p.NQ <= 4 ? launch_t<1, true>(grid, p, s) : launch_t<1, false>(grid, p, s);
}

}  // namespace dd
