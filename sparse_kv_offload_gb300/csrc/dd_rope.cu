// Rotary positions, and appending rows to the cache with the rotation on the way.
//
// The cache is read back by every later step and, in 4 bits, rounded again, so
// the rotation is made independent of how it is computed: the result is the
// bf16 nearest to the exact rotation.  fp32 alone is off where it matters: the
// angle of position 10^5 loses 17 of its 24 bits, and a product rounded to fp32
// falls on the other side of a bf16 tie once in some ten thousand values.  So
//   - a frequency is a 64-bit fraction of a turn, rounded once: position * frequency
//     wraps modulo a turn by itself, off by position * 2^-62 radians at most;
//   - sine and cosine come from 512 stored angles (hi + lo floats) and the angle
//     sum formulas with the remainder |r| <= pi/512, whose series end after
//     r^5 and r^4;
//   - products and sums keep their rounding errors (fma, two-sum), and the last
//     rounding sees them as a sticky bit.
// The sticky bit is needed only next to a tie: a value is first added up to within 2^-22
// of itself, and where both ends of that interval round to the same bf16 number, that is
// the answer.  One lane in a thousand has to go on (26 operations a value instead of 10).
// (With the sines and cosines in fp32 alone the interval is as wide as the larger value's
// error, and a third of the warps had a lane that went on.)
//
// A row is 8 lanes x 16 values: lane i turns up to eight pairs (two 16-byte pieces
// of the row), so a token's sines and cosines are computed once per lane and
// serve all the heads that the warp goes through.
//
// The rotation alone is bound by HBM: four prompts of 4K tokens with 64 heads, half of each
// turned (537 MB), take 84 us, 95% of the copy rate; all of 2K tokens' heads turned (268 MB)
// 48 us, 82%.  (Every value by the sticky path: 231 us; the next head's pieces in registers
// instead of four heads' on their way to shared memory 103 and 59; lanes 0-3 turning all of
// half a row's pairs instead of every lane half of its own 108.)
// Appending 201 MB to bf16 pages takes 39.6 us, 75% (first form 61), bound by the loads that
// 16 warps an SM keep in flight, which is this layout's doing: a thread keeps its sines and cosines,
// 32 registers, for all heads.  Copies to shared memory gain 1 us there, keys and values by
// blocks of their own lose 4.  4 bits are bound by the same 16 warps: they use two thirds of the
// issue slots, most of them for the rounding, and no pipe to its limit (201 MB into 57 MB of pages
// in some 70 us).  Pages in pinned host memory: 131,072 tokens of 8 heads take 2,803 us in bf16
// (191 GB/s, a copy to the host 192) and 852 us in 4 bits (177 GB/s; a row's scales go as
// single bytes).  A step's call of a few rows takes
// 2.6 us (rotation) or 3.1 us (append) on the device, a launch and one row's time.
#include <math.h>

#include "dd_attn.cuh"
#include "dd_kv4.cuh"

namespace dd {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kAhead = 4;               // heads on their way (two: 86 and 53 us, six: 84 and 52)
constexpr int kLut = 512;               // stored angles of a turn
constexpr int kLutOff = 64 * 8;         // table: 64 frequencies, then the stored angles

struct Rope {
  const uint64_t *freq;                 // turns per position * 2^64
  const float4 *lut;                    // {cos hi, sin hi, cos lo, sin lo} * gain
  int rot_dim;                          // 0: no rotation
};

// The eight pairs' cosines and sines at one position, hi + lo.
struct Turn {
  float ch[8], cl[8], sh[8], sl[8];
};

__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
  s = a + b;
  const float t = s - a;
  e = (a - (s - t)) + (b - t);
}

// gain * (cos, sin) of phase / 2^64 turns
__device__ __forceinline__ void cos_sin(uint64_t phase, const float4 *lut, float &ch, float &cl, float &sh,
                                        float &sl) {
  const uint32_t idx = (uint32_t)((phase + (1ull << 54)) >> 55);        // nearest stored angle, 0..512
  const int32_t rem = (int32_t)((int64_t)(phase - ((uint64_t)idx << 55)) >> 23);   // |rem| <= 2^31 - 1: units of 2^-41 turns
  const float rf = (float)rem;
  const float rr = (float)(rem - (int32_t)rf);
  // 2 pi * 2^-41 in two floats
  constexpr double kStep = 6.283185307179586476925286766559 / 2199023255552.0;
  constexpr float kHi = (float)kStep, kLo = (float)(kStep - (double)kHi);
  const float d = rf * kHi;
  const float dl = fmaf(rf, kHi, -d) + fmaf(rf, kLo, rr * kHi);
  const float d2 = d * d;
  const float t = fmaf(d * d2, fmaf(d2, 1.f / 120.f, -1.f / 6.f), dl);     // sin r - d
  const float u = fmaf(d2 * d2, 1.f / 24.f, fmaf(d2, -0.5f, -d * dl));     // cos r - 1
  const float4 a = __ldg(lut + (idx & (kLut - 1)));
  {
    const float p = a.x * d, e = fmaf(a.x, d, -p);
    const float q = fmaf(a.y, u, fmaf(a.x, t, fmaf(a.z, d, e))) + a.w;
    float s, r;
    two_sum(a.y, p, s, r);
    r += q;
    sh = s + r;
    sl = r - (sh - s);
  }
  {
    const float p = -a.y * d, e = fmaf(-a.y, d, -p);
    const float q = fmaf(a.x, u, fmaf(-a.y, t, fmaf(-a.w, d, e))) + a.z;
    float s, r;
    two_sum(a.x, p, s, r);
    r += q;
    ch = s + r;
    cl = r - (ch - s);
  }
}

// bf16 bits of x1 * (ch + cl) + x2 * (sh + sl), x1 and x2 bf16 values: one rounding
__device__ __forceinline__ uint32_t dot2_bf16(float x1, float ch, float cl, float x2, float sh, float sl) {
  const float a = x1 * ch, b = x2 * sh;
  float s, e;
  two_sum(a, b, s, e);
  e += (fmaf(x1, ch, -a) + fmaf(x2, sh, -b)) + fmaf(x1, cl, x2 * sl);
  const float hi = s + e, rest = e - (hi - s);
  uint32_t w = __float_as_uint(hi);
  if (!(fabsf(hi) < INFINITY)) {
    w = __float_as_uint(a + b);     // infinities and NaN: the error terms say nothing
  } else if (rest != 0.f) {
    w -= (rest < 0.f) != (hi < 0.f);    // truncate towards zero, ...
    w |= 1u;                            // ... sticky
  }
  return f2bf(__uint_as_float(w));
}

// The two 16-byte pieces (0..15) of a row that lane i (0..7) holds.  With halves paired:
// a piece of the first half and its partner, the lanes behind them sharing what
// passes through; else pieces i and i + 8, so that a rotation of half the row leaves
// every lane half the work.  Lanes i and i ^ 1 hold both halves of the same two groups of 16,
// and eight lanes load and store whole lines.
template <bool kHalf>
__device__ __forceinline__ void pieces(const Rope &r, int i, int &pa, int &pb) {
  const int n = r.rot_dim / 16;          // lanes that turn (halves paired)
  const bool turns = kHalf && i < n;
  pa = !kHalf || turns ? i : n + i;
  pb = turns ? i + n : i + 8;
}

// The pairs of a lane: 8 i .. of halves, else 4 i .. and 32 + 4 i ..
template <bool kHalf>
__device__ __forceinline__ void make_turn(const Rope &r, int i, int64_t pos, Turn &t) {
  if (kHalf ? i >= r.rot_dim / 16 : i >= r.rot_dim / 8) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (!kHalf && e == 4 && i + 8 >= r.rot_dim / 8) return;
    const int pair = kHalf ? 8 * i + e : 4 * i + (e & 3) + (e >> 2) * 32;
    cos_sin((uint64_t)pos * __ldg(r.freq + pair), r.lut, t.ch[e], t.cl[e], t.sh[e], t.sl[e]);
  }
}

// The pair's rotation with every rounding error kept.  (A function of its own: the common
// path stays short.)
__device__ __noinline__ uint32_t rotate_exactly(float x, float y, float ch, float cl, float sh, float sl) {
  return dot2_bf16(x, ch, cl, -y, sh, sl) | dot2_bf16(y, ch, cl, x, sh, sl) << 16;
}

// x * (ch + cl) + y * (sh + sl), within 2^-23 of itself and 2^-36 of the larger product
__device__ __forceinline__ float dot2_near(float x, float ch, float cl, float y, float sh, float sl) {
  const float p = y * sh;
  return fmaf(x, ch, p) + fmaf(x, cl, fmaf(y, sl, fmaf(y, sh, -p)));
}

// N pairs (x, y) turned by t's E0 .., as bf16 pairs
template <int N, int E0>
__device__ __forceinline__ void rotate_pairs(const Turn &t, const float (&x)[N], const float (&y)[N], uint32_t (&o)[N]) {
  constexpr float kUp = 1.f + 2.384185791015625e-07f, kDown = 1.f - 2.384185791015625e-07f;   // 1 +- 2^-22
  uint32_t near = 0;            // bit e: pair e is next to a tie
  float finite = 0.f;           // NaN once a value is infinite or NaN
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float p = dot2_near(x[e], t.ch[E0 + e], t.cl[E0 + e], -y[e], t.sh[E0 + e], t.sl[E0 + e]);
    const float q = dot2_near(y[e], t.ch[E0 + e], t.cl[E0 + e], x[e], t.sh[E0 + e], t.sl[E0 + e]);
    o[e] = cvt_bf16x2(p * kUp, q * kUp);
    if (o[e] != cvt_bf16x2(p * kDown, q * kDown)) near |= 1u << e;
    finite = fmaf(p, 0.f, fmaf(q, 0.f, finite));
  }
  if (finite != finite) near = 0xFFu;      // the error terms of infinities say nothing
  if (near) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (near >> e & 1u)
        o[e] = rotate_exactly(x[e], y[e], t.ch[E0 + e], t.cl[E0 + e], t.sh[E0 + e], t.sl[E0 + e]);
  }
}

// A piece of neighbouring pairs
template <int E0>
__device__ __forceinline__ void rotate_piece(const Turn &t, uint4 &v) {
  float a[8], x[4], y[4];
  unpack8(v, a);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = a[2 * e], y[e] = a[2 * e + 1];
  uint32_t o[4];
  rotate_pairs<4, E0>(t, x, y, o);
  v = make_uint4(o[0], o[1], o[2], o[3]);
}

// Rotate the lane's two pieces in place.
template <bool kHalf>
__device__ __forceinline__ void rotate(const Rope &r, int i, const Turn &t, uint4 &va, uint4 &vb) {
  if constexpr (kHalf) {
    if (i >= r.rot_dim / 16) return;
    float a[8], b[8];
    unpack8(va, a);
    unpack8(vb, b);
    uint32_t o[8];
    rotate_pairs<8, 0>(t, a, b, o);
    va = make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[4], o[5], 0x5410),
                    __byte_perm(o[6], o[7], 0x5410));
    vb = make_uint4(__byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632), __byte_perm(o[4], o[5], 0x7632),
                    __byte_perm(o[6], o[7], 0x7632));
  } else {
    if (i < r.rot_dim / 8) rotate_piece<0>(t, va);
    if (i + 8 < r.rot_dim / 8) rotate_piece<4>(t, vb);
  }
}

// A thread's 16-byte pieces of the next kAhead heads, on their way to shared memory: no
// thread reads another's, so there is no barrier.
template <int kPieces>
struct Ahead {
  uint4 piece[kAhead][kPieces][kRopeThreads];

  // asks for pieces of head n (none behind the last one); the slot's last reader is done
  template <typename F>
  __device__ __forceinline__ void ask(int n, int heads, F src) {
    if (n < heads) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&piece[n % kAhead][i][threadIdx.x])),
                     "l"(src(i))
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the next head's pieces are here, kAhead - 1 later ones may still be on their way
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
};

struct Rows {          // where the rows of a call lie, in elements
  int64_t b, t, h;
};

// The new rows' token of a lane's row group: its request, row and position.
struct Token {
  bool ok;
  int b;
  int64_t t, pos;
};

__device__ __forceinline__ Token token_of(int64_t n, int B, int T, const int32_t *start_pos, const int32_t *new_len,
                                          int64_t L, int32_t *status) {
  Token k;
  k.ok = n < (int64_t)B * T;
  k.b = k.ok ? (int)(n / T) : 0;
  k.t = k.ok ? n - (int64_t)k.b * T : 0;
  const int len = new_len ? new_len[k.b] : T;
  k.pos = (int64_t)start_pos[k.b] + k.t;
  if (k.ok && (len < 0 || len > T)) {
    set_status(status, DD_ERR_DEVICE_CHECK);
    k.ok = false;
  }
  k.ok = k.ok && k.t < len;
  if (k.ok && (start_pos[k.b] < 0 || k.pos >= L)) {
    set_status(status, DD_ERR_DEVICE_CHECK);
    k.ok = false;
  }
  return k;
}

template <bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) k_rope_rows(Rope r, const uint16_t *__restrict__ x, Rows xs,
                                                            uint16_t *out, Rows os, int B, int T, int H, int heads,
                                                            const int32_t *__restrict__ start_pos,
                                                            const int32_t *__restrict__ new_len, int32_t *status) {
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x & 7;
  const Token k = token_of(((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 3, B, T, start_pos, new_len,
                           INT64_MAX, status);
  if (!k.ok) return;
  int pa, pb;
  pieces<kHalf>(r, i, pa, pb);
  const int h0 = blockIdx.y * heads, h1 = min(H, h0 + heads);
  const uint4 *src = reinterpret_cast<const uint4 *>(x + k.b * xs.b + k.t * xs.t + h0 * xs.h);
  uint4 *dst = reinterpret_cast<uint4 *>(out + k.b * os.b + k.t * os.t + h0 * os.h);
  const int64_t xstep = xs.h / 8, ostep = os.h / 8;
  const int n = h1 - h0;
  __shared__ Ahead<2> ahead;
  uint4 a = src[pa], b = src[pb];
#pragma unroll
  for (int m = 1; m < kAhead; ++m)
    ahead.ask(m, n, [&](int e) { return src + m * xstep + (e ? pb : pa); });
  Turn t;
  make_turn<kHalf>(r, i, k.pos, t);
#pragma unroll 1
  for (int m = 0;;) {
    rotate<kHalf>(r, i, t, a, b);
    ahead.ask(m + kAhead, n, [&](int e) { return src + (m + kAhead) * xstep + (e ? pb : pa); });
    dst[pa] = a;
    dst[pb] = b;
    dst += ostep;
    if (++m == n) break;
    ahead.wait();
    a = ahead.piece[m % kAhead][0][threadIdx.x];
    b = ahead.piece[m % kAhead][1][threadIdx.x];
  }
}

struct AppendP {
  Rope r;
  const uint16_t *k, *v;
  Rows ks, vs;
  int B, T, H, heads, C, cs, shift;       // cs = 1 << shift
  const int32_t *start_pos, *new_len;
  uint8_t *Kh, *Vh, *Khot, *Vhot;
  const int32_t *slot;
  int64_t hot_slots;
  const int32_t *k_exp, *v_exp;
  int32_t *status;
};

// codes and scales of the lane's two pieces into row `row` of the page
__device__ __forceinline__ void store4(uint8_t *page, int row, int pa, int pb, bool even, uint32_t ca, uint32_t cb,
                                       uint32_t sa, uint32_t sb) {
  uint8_t *blk = page + (row >> 4) * kBlk4;
  uint8_t *codes = blk + (row & 15) * 64;
  uint8_t *scales = blk + kBlk4Scales + (row & 15) * 8;
  *reinterpret_cast<uint32_t *>(codes + pa * 4) = ca;
  *reinterpret_cast<uint32_t *>(codes + pb * 4) = cb;
  if (even) {      // (the neighbour lane holds the groups' other halves)
    scales[pa >> 1] = (uint8_t)sa;
    scales[pb >> 1] = (uint8_t)sb;
  }
}

// The largest magnitude of eight bf16 values, as bf16 bits (a NaN's are above infinity's).
__device__ __forceinline__ uint32_t top8(const uint4 &v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(t & 0xFFFFu, t >> 16);
}

// Quantise the lane's two pieces, values divided by 2^e (mul = 2^-e); the other half of
// each piece's group of 16 is the neighbour lane's.  Every lane of the eight takes part.
__device__ __forceinline__ void quantise(const uint4 &va, const uint4 &vb, float mul, unsigned lanes, uint32_t &ca,
                                         uint32_t &cb, uint32_t &sa, uint32_t &sb) {
  uint32_t ta = top8(va), tb = top8(vb);
  const uint32_t both = __shfl_xor_sync(lanes, ta | tb << 16, 1);
  ta = max(ta, both & 0xFFFFu);
  tb = max(tb, both >> 16);
  // (mul is a power of two: the largest value scaled is the largest of the scaled values)
  float ia, ib;
  group_scales(ta, tb, mul, sa, sb, ia, ib);
  float a[8], b[8];
  unpack8(va, a);
  unpack8(vb, b);
  ca = encode8(va, a, ia);
  cb = encode8(vb, b, ib);
}

// A whole group (pieces 2 i and 2 i + 1) by one lane: codes and scale.
__device__ __forceinline__ uint2 quantise_group(const uint4 &va, const uint4 &vb, float mul, uint32_t &scale) {
  const uint32_t top = max(top8(va), top8(vb));
  uint32_t same;
  float inv, inv2;
  group_scales(top, top, mul, scale, same, inv, inv2);
  float a[8], b[8];
  unpack8(va, a);
  unpack8(vb, b);
  return make_uint2(encode8(va, a, inv), encode8(vb, b, inv));
}
__device__ __forceinline__ void store_group(uint8_t *page, int row, int i, uint2 codes, uint32_t scale) {
  uint8_t *blk = page + (row >> 4) * kBlk4;
  *reinterpret_cast<uint2 *>(blk + (row & 15) * 64 + i * 8) = codes;
  blk[kBlk4Scales + (row & 15) * 8 + i] = (uint8_t)scale;
}

template <bool kFour, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) k_append(AppendP p) {
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x & 7;
  const unsigned lanes = 0xFFu << (threadIdx.x & 24);      // the eight lanes of this row
  const Token k = token_of(((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 3, p.B, p.T, p.start_pos, p.new_len,
                           (int64_t)p.C << p.shift, p.status);
  if (!k.ok) return;
  int pa, pb;
  pieces<kHalf>(p.r, i, pa, pb);
  const bool even = (i & 1) == 0;
  const int qa = kFour ? 2 * i : i, qb = kFour ? qa + 1 : i + 8;     // the value row's pieces
  const int c = (int)(k.pos >> p.shift), row = (int)(k.pos & (p.cs - 1));
  const int64_t page_bytes = (int64_t)p.cs * (kFour ? kRow4 : 2 * kD);
  const int h0 = blockIdx.y * p.heads, h1 = min(p.H, h0 + p.heads);
  const uint4 *ksrc = reinterpret_cast<const uint4 *>(p.k + k.b * p.ks.b + k.t * p.ks.t + h0 * p.ks.h);
  const uint4 *vsrc = reinterpret_cast<const uint4 *>(p.v + k.b * p.vs.b + k.t * p.vs.t + h0 * p.vs.h);
  uint4 nka = ksrc[pa], nkb = ksrc[pb], nva = vsrc[qa], nvb = vsrc[qb];
  Turn t;
  make_turn<kHalf>(p.r, i, k.pos, t);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    uint4 ka = nka, kb = nkb;
    const uint4 va = nva, vb = nvb;
    if (h + 1 < h1) {          // the next head's rows are on their way
      ksrc += p.ks.h / 8, vsrc += p.vs.h / 8;
      nka = ksrc[pa], nkb = ksrc[pb], nva = vsrc[qa], nvb = vsrc[qb];
    }
    const int64_t chunk = ((int64_t)k.b * p.H + h) * p.C + c;
    int64_t slot = -1;
    if (p.Khot) {
      slot = p.slot[chunk];
      if (slot < -1 || slot >= p.hot_slots) {
        set_status(p.status, DD_ERR_DEVICE_CHECK);
        slot = -1;
      }
    }
    rotate<kHalf>(p.r, i, t, ka, kb);
    if (kFour) {
      uint32_t kca, kcb, ksa, ksb, vs;
      quantise(ka, kb, pow2i(-head_exp(p.k_exp, h, p.status)), lanes, kca, kcb, ksa, ksb);
      const uint2 vc = quantise_group(va, vb, pow2i(-head_exp(p.v_exp, h, p.status)), vs);
      if (p.Kh) {
        store4(p.Kh + chunk * page_bytes, row, pa, pb, even, kca, kcb, ksa, ksb);
        store_group(p.Vh + chunk * page_bytes, row, i, vc, vs);
      }
      if (slot >= 0) {
        store4(p.Khot + slot * page_bytes, row, pa, pb, even, kca, kcb, ksa, ksb);
        store_group(p.Vhot + slot * page_bytes, row, i, vc, vs);
      }
    } else {
      if (p.Kh) {
        uint4 *kd = reinterpret_cast<uint4 *>(p.Kh + chunk * page_bytes + row * 2 * kD);
        uint4 *vd = reinterpret_cast<uint4 *>(p.Vh + chunk * page_bytes + row * 2 * kD);
        kd[pa] = ka, kd[pb] = kb;
        vd[qa] = va, vd[qb] = vb;
      }
      if (slot >= 0) {
        uint4 *kd = reinterpret_cast<uint4 *>(p.Khot + slot * page_bytes + row * 2 * kD);
        uint4 *vd = reinterpret_cast<uint4 *>(p.Vhot + slot * page_bytes + row * 2 * kD);
        kd[pa] = ka, kd[pb] = kb;
        vd[qa] = va, vd[qb] = vb;
      }
    }
  }
}

Rope rope_of(const dd_rope *r) {
  Rope k{};
  if (r) {
    k.freq = static_cast<const uint64_t *>(r->table);
    k.lut = reinterpret_cast<const float4 *>(static_cast<const uint8_t *>(r->table) + kLutOff);
    k.rot_dim = r->rot_dim;
  }
  return k;
}

// Heads per warp: one while that does not give every SM 16 warps (of 4 tokens), so
// that a step of a few tokens takes one row's time; else 16 at most (by then a token's
// sines and cosines are a tenth of the work), in groups of one size.  A step of 32 rows
// with 32 heads: one head a warp 2.6 us, 16 heads 6.2; a prompt of 4 x 4K tokens with 64
// heads, half of each turned: one 168 us, 8 heads 82.7, 16 heads 83.5, 32 heads 87; all of 4 x 2K
// tokens' 64 heads turned: one 131, 8 heads 52.3, 16 heads 48.1, 32 heads 48.7; append of 4 ragged
// prompts of 8K with 8 heads: one 60.9, 8 heads 39.6; 4-bit append and expansion of 2 x 32K
// tokens with 8 heads: one 168 us, 8 heads 107.
int heads_per_warp(int64_t tokens, int H, int sm_count) {
  const int64_t warps = (tokens + 3) / 4, want = (int64_t)sm_count * 16;
  int64_t groups = (H + 15) / 16;
  if (groups * warps < want) groups = (want + warps - 1) / warps;
  return groups >= H ? 1 : (int)((H + groups - 1) / groups);
}

}  // namespace

cudaError_t launch_rope_rows(const dd_rope *r, const void *x, const int64_t *xs, void *out, const int64_t *os, int B,
                             int T, int H, const int32_t *start_pos, const int32_t *new_len, int sm_count,
                             int32_t *status, cudaStream_t s) {
  const int64_t tokens = (int64_t)B * T;
  const int heads = heads_per_warp(tokens, H, sm_count);
  const int64_t gx = (tokens * 8 + kRopeThreads - 1) / kRopeThreads;
  return launch_k(r->layout == DD_ROPE_HALF ? k_rope_rows<true> : k_rope_rows<false>,
                  dim3((unsigned)gx, (H + heads - 1) / heads), dim3(kRopeThreads), 0, s, rope_of(r),
                  static_cast<const uint16_t *>(x), Rows{xs[0], xs[1], xs[2]}, static_cast<uint16_t *>(out),
                  Rows{os[0], os[1], os[2]}, B, T, H, heads, start_pos, new_len, status);
}

cudaError_t launch_append(const dd_append_args *a, void *kh_dev, void *vh_dev, int B, int Hkv, int C, int cs,
                          int64_t hot_slots, int sm_count, int32_t *status, cudaStream_t s) {
  AppendP p{};
  p.r = rope_of(a->rope);
  p.k = static_cast<const uint16_t *>(a->k);
  p.v = static_cast<const uint16_t *>(a->v);
  p.ks = Rows{a->k_stride[0], a->k_stride[1], a->k_stride[2]};
  p.vs = Rows{a->v_stride[0], a->v_stride[1], a->v_stride[2]};
  p.B = B, p.T = a->T, p.H = Hkv, p.C = C, p.cs = cs;
  p.shift = cs == 16 ? 4 : cs == 32 ? 5 : 6;
  const int64_t tokens = (int64_t)B * a->T;
  p.heads = heads_per_warp(tokens, Hkv, sm_count);
  p.start_pos = a->start_pos, p.new_len = a->new_len;
  p.Kh = static_cast<uint8_t *>(kh_dev), p.Vh = static_cast<uint8_t *>(vh_dev);
  p.Khot = static_cast<uint8_t *>(a->Khot), p.Vhot = static_cast<uint8_t *>(a->Vhot);
  p.slot = a->resident_slot;
  p.hot_slots = hot_slots;
  p.k_exp = a->k_exp, p.v_exp = a->v_exp;
  p.status = status;
  const dim3 grid((unsigned)((tokens * 8 + kRopeThreads - 1) / kRopeThreads), (Hkv + p.heads - 1) / p.heads);
  const bool four = a->format == DD_KV_4BIT, half = a->rope && a->rope->layout == DD_ROPE_HALF;
  return launch_k(four ? half ? k_append<true, true> : k_append<true, false>
                       : half ? k_append<false, true> : k_append<false, false>,
                  grid, dim3(kRopeThreads), 0, s, p);
}

}  // namespace dd

// --------------------------------------------------------------------- host table
// A position is multiplied by the frequency, so a frequency needs all of its 64 bits: from a pow in
// double it would be off by a hundred units of the last one (2^-23 radians at position 2^31),
// and differently with every libm.  So frequencies are worked out in pairs of doubles.
namespace {

struct Wide {            // hi + lo, |lo| at most half a last bit of hi
  double hi, lo;
};

Wide wide_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Wide operator+(Wide a, Wide b) {
  const Wide s = wide_sum(a.hi, b.hi);
  return wide_sum(s.hi, s.lo + (a.lo + b.lo));
}
Wide operator-(Wide a) { return {-a.hi, -a.lo}; }
Wide operator*(Wide a, Wide b) {
  const double p = a.hi * b.hi, e = fma(a.hi, b.hi, -p);
  return wide_sum(p, e + (a.hi * b.lo + a.lo * b.hi));
}
Wide operator/(Wide a, Wide b) {
  const double q = a.hi / b.hi;
  const Wide rest = a + -(b * Wide{q, 0.0});
  return wide_sum(q, (rest.hi + rest.lo) / b.hi);
}

// a^n times 2^-e, the powers of two kept apart so that nothing overflows
Wide wide_power(Wide a, int n, int &e) {
  Wide r{1.0, 0.0};
  int ea = 0;
  e = 0;
  auto scale = [](Wide &x, int &ex) {
    int k;
    frexp(x.hi, &k);
    x = {ldexp(x.hi, -k), ldexp(x.lo, -k)};
    ex += k;
  };
  for (scale(a, ea); n; n >>= 1) {
    if (n & 1) {
      r = r * a;
      e += ea;
      scale(r, e);
    }
    a = a * a;
    ea *= 2;
    scale(a, ea);
  }
  return r;
}

// base^(-i/n), 0 <= i < n <= 64: from pow's answer y by Newton's steps on y^n base^i = 1 (an error of
// 2^-44 of y becomes one of 2^-83, and that one vanishes)
Wide wide_root(double base, int i, int n) {
  Wide y{pow(base, -(double)i / n), 0.0};
  for (int step = 0; step < 2; ++step) {
    int ey, eb;
    const Wide p = wide_power(y, n, ey), b = wide_power({base, 0.0}, i, eb), one = p * b;
    const Wide off = Wide{ldexp(one.hi, ey + eb), ldexp(one.lo, ey + eb)} + Wide{-1.0, 0.0};
    y = y + -(y * (off / Wide{(double)n, 0.0}));
  }
  return y;
}

Wide clamp01(Wide x) { return x.hi < 0.0 ? Wide{0.0, 0.0} : x.hi >= 1.0 ? Wide{1.0, 0.0} : x; }

}  // namespace

static bool rope_params_ok(const dd_rope_params *p) {
  if (!p || p->rot_dim < 32 || p->rot_dim > dd::kD || p->rot_dim % 32) return false;
  if (!(p->base > 1.0) || !isfinite(p->base) || !isfinite(p->gain)) return false;
  if (p->scaling < DD_ROPE_PLAIN || p->scaling > DD_ROPE_BY_WAVELENGTH) return false;
  if (p->scaling != DD_ROPE_PLAIN && !(p->factor >= 1.0 && isfinite(p->factor))) return false;
  if (p->scaling >= DD_ROPE_BY_PARTS &&
      !(p->orig_len > 0.0 && isfinite(p->orig_len) && p->beta_slow > 0.0 && p->beta_fast > p->beta_slow &&
        isfinite(p->beta_fast)))
    return false;
  return true;
}

extern "C" dd_status dd_rope_table(const dd_rope_params *p, void *table) {
  if (!rope_params_ok(p) || !table) return DD_ERR_INVALID_ARG;
  const double pi2 = 6.283185307179586476925286766559;
  const Wide kPerRadian{0.15915494309189535, -9.839338337591243e-18};     // 1 / (2 pi)
  const int n = p->rot_dim / 2;
  double lo = 0, hi = 0;
  if (p->scaling == DD_ROPE_BY_PARTS) {
    const double a = p->rot_dim * log(p->orig_len / (p->beta_fast * pi2)) / (2.0 * log(p->base));
    const double b = p->rot_dim * log(p->orig_len / (p->beta_slow * pi2)) / (2.0 * log(p->base));
    lo = floor(a) > 0.0 ? floor(a) : 0.0;
    hi = ceil(b) < p->rot_dim - 1.0 ? ceil(b) : p->rot_dim - 1.0;
  }
  uint64_t *freq = static_cast<uint64_t *>(table);
  for (int i = 0; i < 64; ++i) {
    freq[i] = 0;
    if (i >= n) continue;
    const Wide whole{1.0, 0.0}, factor{p->factor, 0.0};
    Wide f = wide_root(p->base, i, n);
    if (p->scaling == DD_ROPE_LINEAR) {
      f = f / factor;
    } else if (p->scaling == DD_ROPE_NTK) {      // (base * factor^(n/(n-1)))^(-i/n)
      f = f * wide_root(p->factor, i, n - 1);
    } else if (p->scaling == DD_ROPE_BY_PARTS) {
      const Wide r = clamp01(Wide{i - lo, 0.0} / Wide{hi - lo > 1e-3 ? hi - lo : 1e-3, 0.0});
      f = f * (whole + -r) + f / factor * r;
    } else if (p->scaling == DD_ROPE_BY_WAVELENGTH) {
      // (the borders first: between them the quotient is one of numbers of a size)
      const Wide turns = Wide{p->orig_len, 0.0} * f * kPerRadian;
      const Wide r = turns.hi < p->beta_slow    ? Wide{0.0, 0.0}
                     : turns.hi >= p->beta_fast ? whole
                                                : clamp01((turns + Wide{-p->beta_slow, 0.0}) /
                                                          wide_sum(p->beta_fast, -p->beta_slow));
      f = f * r + f / factor * (whole + -r);
    }
    // turns per position, times 2^64 (f <= 1, so below 2^62), to the nearest integer
    const Wide t = f * kPerRadian;
    const double v = ldexp(t.hi, 64), th = floor(v), tl = floor((v - th) + ldexp(t.lo, 64) + 0.5);
    freq[i] = (uint64_t)th + (uint64_t)(int64_t)tl;
  }
  const double gain =
      p->gain > 0.0 ? p->gain : p->scaling == DD_ROPE_BY_PARTS ? 0.1 * log(p->factor) + 1.0 : 1.0;
  float *lut = reinterpret_cast<float *>(static_cast<uint8_t *>(table) + dd::kLutOff);
  for (int i = 0; i < dd::kLut; ++i) {
    const double c = gain * cos(pi2 * i / dd::kLut), s = gain * sin(pi2 * i / dd::kLut);
    lut[4 * i + 0] = (float)c;
    lut[4 * i + 1] = (float)s;
    lut[4 * i + 2] = (float)(c - (double)(float)c);
    lut[4 * i + 3] = (float)(s - (double)(float)s);
  }
  return DD_OK;
}
