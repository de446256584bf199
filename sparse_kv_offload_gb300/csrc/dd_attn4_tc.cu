// Attention over 4-bit pages on the fifth-generation tensor cores, for more than 16
// query vectors per KV head.
//
// With many query vectors the products, not the bytes, bound the mma.sync kernel
// (dd_attn4.cu), and each 16 of them would decode a unit's pages again.  Here a page is
// decoded once, into shared memory, for up to 64 query vectors, and the accumulators
// live in tensor memory.  One CTA per SM; a tile is 128 rows (eight blocks), so that a
// tile's fixed costs (barriers, waits, the vote) are paid half as often as with 64:
//   warp 12     asks for a tile's blocks (bulk copies into a ring of three tiles)
//   warps 8-11  decode two blocks each: fp16 K and V (a code times its scale is exact), in
//               the 128-byte-swizzled layout that the products read; K has one buffer,
//               free again after S, V two
//   warp 13     S = Q K^T (M = 64 query vectors, N = 128 rows, K = 128), double-buffered in
//               tensor memory, and O += P V (N = 128 columns, K = 128 rows) with both parts
//               of P as one operand of 128 rows, which takes no longer than 64
//   warps 0-7   softmax, four threads a query vector (the M = 64 layout: row r in lane 32 (r
//               / 16) + r % 16); P goes to shared memory as two fp16 parts (22 bits)
// The tensor cores truncate when they add (the sums of 8,192 tiles are off by 1.5e-5): they
// add up at most kFold tiles (1e-6); then, and where a score exceeds the softmax's reference
// by 2^8, the softmax threads take O over into fp32 registers, where additions round to
// nearest, and the next product overwrites it.  What truncation is left there and in the
// 128 terms of a score, P's 22 bits and an exponential good to 2^-22 (ex2.approx) leave up to
// 2.3e-6 of the output (128K rows, 40 query vectors; plain fp32 4.2e-6), and on some short unions up
// to 1.8 times plain fp32's error (1.1e-6 for 6.2e-7).
//
// Bound by the softmax threads' chain per tile (some 3,200 cycles, most of them latency: the
// loads of S 900, the exponentials and P's stores 900, two barriers, O's look 400), which
// the products (1,024, issued in 720) and the decoding (2,500) run beside, and by the ends of
// runs, a quarter of the time here.  32B-class layer, five queries (171 MB of pages, floor 25 us):
// the mma.sync kernel in groups of 16 215 us, 64-row tiles 182, 128-row tiles 151, both
// parts of P in one operand and O taken over every eight tiles instead of two 141, the
// products issued by an elected thread of a whole warp, which keeps the descriptors in uniform
// registers (lane 0 alone took 1,730 cycles for a tile's 16), 133.  Not kept: sixteen softmax
// warps (80 registers; 1-3% gained with 40 or more query vectors, 5% lost with 20), eight
// decoding warps (96 registers, -10%) or two blocks decoded at once (160 us: the softmax waits
// for their shared-memory traffic), a second buffer for P (146), two groups of four softmax warps on
// alternate tiles (184), P from the old reference with the vote at its end (136).
#include "dd_attn4.cuh"

namespace dd {

namespace {

constexpr int kSoft = 8;                            // softmax warps
constexpr int kDecode = 4;                          // decoding warps
constexpr int kTcThreads = (kSoft + kDecode + 2) * 32;
constexpr int kTcM = 64;
constexpr int kBlocks = 8;                          // blocks of a tile
constexpr int kRaw = 3, kK = 1, kV = 2;             // tiles: as they are, and decoded (K's buffer is free after S)
constexpr int kRawBytes = kBlocks * 2 * kBlk4;
constexpr int kHalf = 64 * 128;                     // 64 rows of 64 fp16 values (queries, P)
constexpr int kTileHalf = 128 * 128;                // 128 rows of 64 fp16 values (K, V)
constexpr int kKvBytes = 2 * kTileHalf;             // lo, hi
constexpr int kMeta = 8;                            // tiles' records
constexpr int kFold = 8;
constexpr uint32_t kTmemCols = 512;                 // S: 2 x 128 columns, O: 128
constexpr size_t kTcSmem = 1024 + (size_t)(kK + kV) * kKvBytes + 2 * kHalf + 4 * kHalf + (size_t)kRaw * kRawBytes;

// kind::f16 instruction descriptor with fp16 A and B: fp32 accumulator, B's major-ness, N, M
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One thread of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSoft * 32) : "memory"); }

// A thread's 32 columns of S (two loads, one wait): threads 0-15 of the warp at c, 16-31 at
// c + 32, of lanes 0-15 of the warp's quarter.
__device__ __forceinline__ void tmem_ld_s(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 32;"
        : "=r"(r[16 * h]), "=r"(r[16 * h + 1]), "=r"(r[16 * h + 2]), "=r"(r[16 * h + 3]), "=r"(r[16 * h + 4]),
          "=r"(r[16 * h + 5]), "=r"(r[16 * h + 6]), "=r"(r[16 * h + 7]), "=r"(r[16 * h + 8]), "=r"(r[16 * h + 9]),
          "=r"(r[16 * h + 10]), "=r"(r[16 * h + 11]), "=r"(r[16 * h + 12]), "=r"(r[16 * h + 13]),
          "=r"(r[16 * h + 14]), "=r"(r[16 * h + 15])
        : "r"(taddr + 16 * h));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// acc = (acc + a thread's 32 columns of O) * factor.  Lanes 0-15 of the quarter hold the sums
// of P's first part, lanes 16-31 those of its second: a thread reads 64 columns of its
// lane, 16 at a time, and gives half of them away.
__device__ __forceinline__ void tmem_add_o(uint32_t taddr, float (&acc)[32], float factor, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float a[16], b[16];
    tmem_ld32x32b_x16(taddr + 16 * h, a);
    tmem_ld32x32b_x16(taddr + 32 + 16 * h, b);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float keep = lane < 16 ? a[e] : b[e], give = lane < 16 ? b[e] : a[e];
      acc[16 * h + e] = (acc[16 * h + e] + (keep + __shfl_xor_sync(0xffffffffu, give, 16))) * factor;
    }
  }
}

// A block's 16 rows of 128 values -> fp16, 16-byte pieces of 8 values: a lane takes piece c
// of rows 2 it + lane / 16.  dst: the tile's lo half at the block's first row.  Scales of V's
// rows behind the end, which may hold anything, and NaN ones (0 * NaN would reach every
// query) count as 0.
template <bool kValues>
__device__ __forceinline__ void decode_block(uint32_t raw, uint32_t dst, int rows, int lane) {
  const int c = lane & 15, half = lane >> 4;
  const uint32_t codes = raw + half * 64 + c * 4, scales = raw + kBlk4Scales + half * 8 + (c >> 1);
  dst += (uint32_t)((c >> 3) * kTileHalf + half * 128);
  uint32_t w[8], s[8];   // all loads first: the eight pieces' chains then overlap
#pragma unroll
  for (int it = 0; it < 8; ++it) s[it] = lds8(scales + it * 16), w[it] = lds32(codes + it * 128);
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int row = 2 * it + half;
    if (kValues && (row >= rows || (s[it] & 0x7Fu) == 0x7Fu)) s[it] = 0;
    const uint32_t s2 = e4m3x2_to_half2(s[it] * 0x101u);
    uint32_t h[4];
    e2m1x8_to_half2(w[it], h);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = hmul2_u32(h[e], s2);
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (uint32_t)(it * 256 +
                                                                              (((c & 7) ^ (row & 7)) << 4))),
                 "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                 : "memory");
  }
}

// Groups of 16 columns (bits) in which one of V's first `rows` rows is NaN: the warp's 16
// bytes x 8 of scales, a word a lane.
__device__ __forceinline__ uint32_t nan_groups(uint32_t raw_v, int rows, int lane) {
  const uint32_t w = lds32(raw_v + kBlk4Scales + lane * 4);      // row lane / 2, groups 4 (lane & 1) ..
  const uint32_t n = (lane >> 1) < rows ? (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) : 0u;
  if (!__any_sync(0xffffffffu, n != 0u)) return 0u;
  uint32_t bits = (n >> 7 & 1u) | (n >> 14 & 2u) | (n >> 21 & 4u) | (n >> 28 & 8u);
  bits <<= 4 * (lane & 1);
  return __reduce_or_sync(0xffffffffu, bits);
}

__global__ void __launch_bounds__(kTcThreads, 1) k_attn4_tc(const __grid_constant__ Attn4Params p) {
  extern __shared__ uint8_t smem_raw[];
  // the swizzle pattern is anchored at 1024-byte boundaries
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t kv0 = smem_u32(smem), v0 = kv0 + kK * kKvBytes;     // [kK][kKvBytes], [kV][kKvBytes]
  const uint32_t q0s = v0 + kV * kKvBytes;                           // [2 halves][64 rows][128 B]
  const uint32_t p0 = q0s + 2 * kHalf;                               // [2 halves][128 rows][128 B]
  const uint32_t raw0 = p0 + 4 * kHalf;                              // [kRaw][kBlocks][K, V]
  // a run's sums, in P's place once its last product is done: [64 rows][32 pieces of 4
  // columns], piece c of row r at c ^ (r & 31)
  float4 *join = reinterpret_cast<float4 *>(smem + (p0 - kv0));
  __shared__ PlanSmem plan;
  __shared__ __align__(8) uint64_t bars[2 * kRaw + 2 * kK + 2 * kV + 6];
  __shared__ uint4 s_tails[2 * kMaxNq * 16];
  __shared__ __align__(16) uint32_t s_meta[kMeta][kBlocks], s_nan[kMeta][kBlocks];
  __shared__ float s_back[kTcM], s_m[kTcM], s_l[kTcM], s_red[2][kTcM];
  __shared__ uint32_t s_tmem;
  __shared__ int s_over, s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const Attn4Args &a = p.a;
  const uint32_t raw_full = smem_u32(bars), raw_empty = raw_full + 8 * kRaw;
  const uint32_t k_full = raw_empty + 8 * kRaw, k_empty = k_full + 8 * kK, v_full = k_empty + 8 * kK,
                 v_empty = v_full + 8 * kV;
  const uint32_t s_full = v_empty + 8 * kV, pv_done = s_full + 16, p_ready = pv_done + 8, q_full = p_ready + 8;
  const uint32_t mma_done = q_full + 8;
  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) mbar_init(raw_full + 8 * i, kBlocks), mbar_init(raw_empty + 8 * i, kDecode);
    for (int i = 0; i < kK; ++i) mbar_init(k_full + 8 * i, kDecode), mbar_init(k_empty + 8 * i, 1);
    for (int i = 0; i < kV; ++i) mbar_init(v_full + 8 * i, kDecode), mbar_init(v_empty + 8 * i, 1);
    mbar_init(s_full, 1), mbar_init(s_full + 8, 1);
    mbar_init(pv_done, 1);
    mbar_init(p_ready, 1);
    mbar_init(q_full, 1);
    mbar_init(mma_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  Slice<kTcThreads, 1, 3> slice;
  if (!slice.open(p, plan)) return;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem, tmem_o = tmem + 256;
  const uint32_t all_q = (1u << a.n_q) - 1u;

  // Every role walks the same tiles and numbers them alike.  A wait that runs out (2 s)
  // only ends that thread's waiting: the barriers below are still met by all.
  int t = 0, run_no = 0;
  bool alive = true;
  auto wait = [&](uint32_t bar, int parity) {
    if (alive && !mbar_wait(bar, (uint32_t)parity & 1u, a.status)) alive = false;
  };

  for (int w0 = 0;; w0 += kMaxRuns) {
    int wlo, whi;
    const int n_runs = slice.list(p, plan, w0, wlo, whi);
    const Run *runs = plan.runs;
    const int n_tiles = whi - wlo;

    if (slice.dead) {
      // an error is pending: no work, but the counts of shared units go on
      if (tid == 0)
        for (int r = 0; r < n_runs; ++r)
          if (runs[r].cta0 != runs[r].cta1) arrive_at_unit(p, runs[r], true);
    } else if (warp == kSoft + kDecode) {
      // ------------------------------------------------------------- loads
      for (int i0 = 0; i0 < n_tiles; i0 += 4) {
        // lane 8 k + h: block h of tile i0 + k
        BlockRef ref = {0, 0u};
        const int x = wlo + i0 + (lane >> 3);
        if (x < whi) {
          int r = 0;
#pragma unroll
          for (int step = kMaxRuns / 2; step > 0; step >>= 1)
            if (r + step < n_runs && runs[r + step].start <= x) r += step;
          ref = look_at(p, load_entry(p, runs[r], kBlocks * (x - runs[r].start) + (lane & 7), all_q), slice.staged, all_q);
        }
        for (int k = 0; k < 4 && i0 + k < n_tiles; ++k, ++t) {
          const int st = t % kRaw;
          if (t >= kRaw) wait(raw_empty + 8 * st, t / kRaw - 1);
          __syncwarp();
          if ((lane >> 3) == k) {
            s_meta[t % kMeta][lane & 7] = ref.meta;      // (the arrival below releases it)
            if (ref.meta && alive)
              load_block(p, ref, raw0 + st * kRawBytes + (lane & 7) * 2 * kBlk4, raw_full + 8 * st);
            else
              mbar_arrive(raw_full + 8 * st);
          }
        }
      }
    } else if (warp >= kSoft && warp < kSoft + kDecode) {
      // ------------------------------------------------------------ decoding
      const int w = warp - kSoft;
      for (int i = 0; i < n_tiles; ++i, ++t) {
        const int st = t % kRaw, kb = t % kK, vb = t % kV;
        wait(raw_full + 8 * st, t / kRaw);
        if (t >= kK) wait(k_empty + 8 * kb, t / kK - 1);
        __syncwarp();
#pragma unroll 1
        for (int blk = w; blk < kBlocks; blk += kDecode) {
          const uint32_t raw = raw0 + st * kRawBytes + blk * 2 * kBlk4;
          const int rows = (int)(s_meta[t % kMeta][blk] >> 8) & 31;
          const uint32_t nan = nan_groups(raw + kBlk4, rows, lane);
          if (lane == 0) s_nan[t % kMeta][blk] = nan;
          decode_block<false>(raw, kv0 + kb * kKvBytes + blk * 16 * 128, 16, lane);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + 8 * kb);
        if (t >= kV) wait(v_empty + 8 * vb, t / kV - 1);
        __syncwarp();
#pragma unroll 1
        for (int blk = w; blk < kBlocks; blk += kDecode) {
          const uint32_t raw = raw0 + st * kRawBytes + (blk * 2 + 1) * kBlk4;
          const int rows = (int)(s_meta[t % kMeta][blk] >> 8) & 31;
          decode_block<true>(raw, v0 + vb * kKvBytes + blk * 16 * 128, rows, lane);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v_full + 8 * vb);
          mbar_arrive(raw_empty + 8 * st);
        }
      }
    } else if (warp == kSoft + kDecode + 1) {
      // ------------------------------------------------------------ products
      // (the whole warp waits and counts, so that what the products are told is uniform)
      {
        // (descriptors hold addresses in 16-byte units: a step adds a constant)
        constexpr uint32_t id_s = idesc_f16(kTcM, 128, 0), id_o = idesc_f16(128, 128, 1);
        const uint64_t q_desc = smem_desc_sw128(q0s, 16, 1024), k_desc = smem_desc_sw128(kv0, 16, 1024);
        const uint64_t p_desc = smem_desc_sw128(p0, 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(v0, kTileHalf, 1024);
        auto issue_pv = [&](int u) {
          wait(v_full + 8 * (u % kV), u / kV);
          wait(p_ready, u);
          tc_fence_after();
          if (!__all_sync(0xffffffffu, alive)) return;
          const uint64_t vb = v_desc + (uint32_t)((u % kV) * (kKvBytes / 16));
          const bool over = __shfl_sync(0xffffffffu, s_over, 0) != 0;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma(tmem_o, p_desc + ((ks >> 2) * kTileHalf + (ks & 3) * 32) / 16, vb + ks * 16 * 128 / 16, id_o,
                     !(over && ks == 0));
            tc_commit(v_empty + 8 * (u % kV));
            tc_commit(pv_done);
          }
        };
        int x = wlo;
        for (int r = 0; r < n_runs; ++r, ++run_no) {
          const int end = min(whi, runs[r].end);
          wait(q_full, run_no);
          for (; x < end; ++x, ++t) {
            wait(k_full + 8 * (t % kK), t / kK);
            tc_fence_after();
            if (__all_sync(0xffffffffu, alive) && elect_one()) {
              // the softmax threads are done with S(t - 2): P(t - 2) was ready
              const uint64_t kb = k_desc + (uint32_t)((t % kK) * (kKvBytes / 16));
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                tc_mma(tmem + (t & 1) * 128, q_desc + ((ks >> 2) * kHalf + (ks & 3) * 32) / 16,
                       kb + ((ks >> 2) * kTileHalf + (ks & 3) * 32) / 16, id_s, ks > 0);
              tc_commit(s_full + 8 * (t & 1));
              tc_commit(k_empty + 8 * (t % kK));
            }
            // S of this tile runs beside the softmax of the one before, its P V comes after it
            if (x > max(wlo, runs[r].start)) issue_pv(t - 1);
            if (x + 1 == end) issue_pv(t);
          }
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------- softmax
      const int wq = warp & 3, wc = warp >> 2, sub = lane >> 4;
      const int row = 16 * wq + (lane & 15);             // query vector
      const int bi = 2 * wc + sub;                       // 32 columns of S (blocks 2 bi, 2 bi + 1) and of O
      const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
      const bool active = row < p.NQ, some = 16 * wq < p.NQ;     // some: of this warp's query vectors
      const int j = active ? row / p.G : 31;
      const float sl2 = a.softmax_scale * 1.4426950408889634f;
      for (int r = 0; r < n_runs; ++r) {
        const Run &run = runs[r];
        const int n = min(whi, run.end) - max(wlo, run.start);
        stage_tails(p, run, s_tails, tid, kSoft * 32);
        {
          // the queries: four threads a query vector, 32 values each
          const int qv = tid >> 2, part = tid & 3;
          uint4 w[4];
          if (qv < p.NQ) {
            const uint4 *src =
                reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + out_row(p, run.unit, qv) + 32 * part);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = src[e];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = make_uint4(0u, 0u, 0u, 0u);
          }
          uint32_t f[16];
          float back;
          query_fragments(w, f, back);
          if (part == 0) s_back[qv] = score_factor(back, sl2 * pow2i(run.ke));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = 4 * part + e;
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                             q0s + (uint32_t)((c >> 3) * kHalf + qv * 128 + (((c & 7) ^ (qv & 7)) << 4))),
                         "r"(f[4 * e]), "r"(f[4 * e + 1]), "r"(f[4 * e + 2]), "r"(f[4 * e + 3])
                         : "memory");
          }
        }
        cp_async_wait_all();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        soft_barrier();
        if (tid == 0) mbar_arrive(q_full);

        const float mul = s_back[row];
        float m = -INFINITY, l = 0.f, oacc[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) oacc[e] = 0.f;
        int since = 0;                                   // tiles in O since it was taken over
        for (int i = 0; i < n; ++i, ++t) {
          wait(s_full + 8 * (t & 1), t >> 1);
          __syncwarp();
          tc_fence_after();
          float x[32], pm = -INFINITY;
          if (some) {
            tmem_ld_s(tmem + lane_base + (t & 1) * 128 + 64 * wc, x);
            // (the mask comes after the factor, which may be 0)
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] *= mul;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t meta = s_meta[t % kMeta][2 * bi + h];
              const int rows = (meta & 255u) >> j & 1u ? (int)(meta >> 8) & 31 : 0;
              if (rows < 16) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (e >= rows) x[16 * h + e] = -INFINITY;
              }
            }
            float m8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) m8[e] = fmaxf(fmaxf(x[e], x[e + 8]), fmaxf(x[e + 16], x[e + 24]));
#pragma unroll
            for (int e = 0; e < 4; ++e) m8[e] = fmaxf(m8[e], m8[e + 4]);
            pm = fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3]));
            pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 16));
            if (sub == 0) s_red[wc][row] = pm;
          }
          // one barrier exchanges the halves' maxima and votes on a new reference
          uint32_t any;
          asm volatile(
              "{\n .reg .pred q, r;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred r, 1, %2, q;\n selp.u32 %0, 1, 0, r;\n}\n"
              : "=r"(any)
              : "r"((uint32_t)(pm > highest_for(m))), "n"(kSoft * 32)
              : "memory");
          const float mx = some ? fmaxf(s_red[0][row], s_red[1][row]) : -INFINITY;
          float factor = 1.f;
          if (mx > highest_for(m)) {
            const float nm = mx - kHead;
            factor = weight_of(m, nm);
            m = nm;
          }
          const bool fold = i > 0 && (any || since == kFold);
          // P's and O's last reader and writer: PV(t - 1)
          if (t > 0) wait(pv_done, t - 1);
          if (fold && some) {
            __syncwarp();
            tc_fence_after();
            tmem_add_o(tmem_o + lane_base + 64 * wc, oacc, factor, lane);
            l *= factor;
          }
          if (fold) since = 0;
          {
            const uint4 n0 = *reinterpret_cast<const uint4 *>(s_nan[t % kMeta]);
            const uint4 n1 = *reinterpret_cast<const uint4 *>(s_nan[t % kMeta] + 4);
            if ((n0.x | n0.y | n0.z | n0.w | n1.x | n1.y | n1.z | n1.w) != 0u) {
              // NaN groups of V: NaN for the queries that see their block
#pragma unroll 1
              for (int blk = 0; blk < kBlocks; ++blk) {
                const uint32_t nan = s_nan[t % kMeta][blk];
                if (!((s_meta[t % kMeta][blk] & 255u) >> j & 1u)) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (nan >> (2 * bi + h) & 1u) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) oacc[16 * h + e] = NAN;
                  }
              }
            }
          }
          if (active) {
            // a query without a row so far: -inf - 0 gives weight 0, and a NaN passes
            const float base = m == -INFINITY ? 0.f : m;
            const uint32_t ph = p0 + (bi >> 1) * kTileHalf + (32 * wq + (lane & 15)) * 128;     // the second part 16 rows on
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t hi[4], lo[4];
              float sum = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float u = ex2_approx(x[8 * c + 2 * e] - base), v = ex2_approx(x[8 * c + 2 * e + 1] - base);
                sum += u + v;
                hi[e] = cvt_f16x2(u, v);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi[e]));
                lo[e] = cvt_f16x2(u - f.x, v - f.y);
              }
              l += sum;
              const uint32_t off = (uint32_t)((((bi & 1) * 4 + c) ^ (row & 7)) << 4);
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(ph + off), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]),
                           "r"(hi[3])
                           : "memory");
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(ph + 16 * 128 + off), "r"(lo[0]), "r"(lo[1]),
                           "r"(lo[2]), "r"(lo[3])
                           : "memory");
            }
          }
          if (tid == 0) s_over = i == 0 || fold;
          ++since;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc_fence_before();
          soft_barrier();
          if (tid == 0) mbar_arrive(p_ready);
        }

        // ------------------------------------------------- the run's sums
        wait(pv_done, t - 1);
        __syncwarp();
        tc_fence_after();
        tmem_add_o(tmem_o + lane_base + 64 * wc, oacc, 1.f, lane);
        tc_fence_before();      // O is read before the next run's first product overwrites it
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (sub == 0) s_red[wc][row] = l;
        if (bi == 0) s_m[row] = m;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          join[row * 32 + ((8 * bi + e) ^ (row & 31))] =
              make_float4(oacc[4 * e], oacc[4 * e + 1], oacc[4 * e + 2], oacc[4 * e + 3]);
        soft_barrier();
        if (tid < kTcM) s_l[tid] = s_red[0][tid] + s_red[1][tid];
        soft_barrier();
        const bool shared = run.cta0 != run.cta1;
        const float vmul = pow2i(run.ve);
        const uint2 *tails = reinterpret_cast<const uint2 *>(s_tails);
        auto query_of = [&](int k) {
          return a.k_tail ? *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) +
                                                             out_row(p, run.unit, k) + 4 * lane)
                          : make_uint2(0u, 0u);
        };
#pragma unroll 2
        for (int k = warp; k < p.NQ; k += kSoft) {
          const float4 v = join[k * 32 + (lane ^ (k & 31))];
          const Part s = {s_m[k], s_l[k], make_float4(v.x * vmul, v.y * vmul, v.z * vmul, v.w * vmul)};
          if (!shared) {
            finish(p, run.unit, k, s, query_of(k), tails, lane);
          } else {
            const int64_t at = ((int64_t)blockIdx.x + run.unit) * p.group_q + k;
            *reinterpret_cast<float4 *>(p.part_o + at * kD + 4 * lane) = s.o;
            if (lane == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(s.m, s.l);
          }
        }
        soft_barrier();
        if (shared) {
          // the barrier above orders the CTA's parts before the count, the one below the count before the reads
          if (tid == 0) s_last = arrive_at_unit(p, run, false);
          soft_barrier();
          if (s_last)
            for (int k = warp; k < p.NQ; k += kSoft)
              finish(p, run.unit, k, combine_parts(p, run, k, lane), query_of(k), tails, lane);
          soft_barrier();       // s_last and the tails are read
        }
      }
    }
    if (whi >= slice.hi) break;
  }
  // (the decoding warps have waited for every copy, unless a wait has run out)
  if (warp == kSoft + kDecode) ring_drain(raw_full, kRaw, (uint32_t)max(t - kRaw, 0), (uint32_t)t, lane, a.status);
  // every product issued is done before the tensor memory is freed
  if (warp == kSoft + kDecode + 1 && elect_one()) {
    tc_commit(mma_done);
    mbar_wait(mma_done, 0, a.status);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace

cudaError_t launch_attn4_tc(int grid, const Attn4Params &p, cudaStream_t s) {
  cudaError_t e = set_dyn_smem((const void *)k_attn4_tc, kTcSmem);
  if (e != cudaSuccess) return e;
  return launch_k(k_attn4_tc, dim3(grid), dim3(kTcThreads), kTcSmem, s, p);
}

}  // namespace dd
