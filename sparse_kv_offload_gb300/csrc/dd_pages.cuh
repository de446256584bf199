// Shared parts of the kernels that read a paged cache through lists of chunks
// (attention of new tokens, dd_extend.cu; chunk weights, dd_weights.cu): the arguments
// they have in common, requests and lists as they are read from device memory,
// tensor-memory and packed-float helpers, and the host makers of their tensor maps.
#ifndef DD_PAGES_CUH_
#define DD_PAGES_CUH_

#include <limits.h>

#include "dd_attn.cuh"

namespace dd {

constexpr int kTileKeys = 128;                    // keys of a tile
constexpr int kTileHalfBytes = 128 * 128;         // 128 rows of 64 bf16 values, 128-byte swizzle
constexpr int kTileBytes = 2 * kTileHalfBytes;

// Queries, lists and pools, as both kernels take them.
struct PagesArgs {
  const int32_t *start_pos, *new_len;             // [B]; new_len null: T
  const int32_t *union_idx, *union_slot;          // [B,Hkv,umax]
  const int32_t *union_cnt, *miss_count;          // [B,Hkv]; [1] or null
  int B, T, Hq, Hkv, G, cs, cs_log, C, umax;      // cs = 2^cs_log
  int tt;                                         // tokens of a tile of query rows: tt * G <= 128
  int64_t hot_slots, max_misses;
  float scale, sl2;                               // softmax scale, and times log2 e
  // The status word stops a launch where an error was pending before it.  What the launch itself finds goes to
  // another word, which its last CTA moves there: CTAs that start later do their work all the same.
  int32_t *status, *raised;
};

struct Request {
  int start, len;                                 // a request that is out of range has no tokens
};

__device__ __forceinline__ Request check_request(const PagesArgs &a, int start, int len) {
  if (start < 0 || len < 0 || len > a.T || (int64_t)start + len > (int64_t)a.C * a.cs) {
    set_status(a.raised, DD_ERR_DEVICE_CHECK);
    return {0, 0};
  }
  return {start, len};
}

__device__ __forceinline__ Request load_request(const PagesArgs &a, int b) {
  return check_request(a, a.start_pos[b], a.new_len ? a.new_len[b] : a.T);
}

__device__ __forceinline__ int check_count(const PagesArgs &a, int n) {
  if (n < 0 || n > a.umax) {
    set_status(a.raised, DD_ERR_DEVICE_CHECK);
    return 0;
  }
  return n;
}

__device__ __forceinline__ int load_count(const PagesArgs &a, int unit) { return check_count(a, a.union_cnt[unit]); }

// Entry e of a unit's list: the chunk's slot (hot: slot, staged: -(m+1)) and the position of
// its first row; INT_MAX where there is none or it is out of range (the slot is then looked at no more).
struct Entry {
  int slot, pos;
};

// As the list holds it: loaded ahead of its use and looked at then (a check behind the load would wait for it).
struct RawEntry {
  int slot, idx;
};

__device__ __forceinline__ RawEntry fetch_entry(const PagesArgs &a, int64_t list, int e, int n) {
  if (e >= n) return {0, 0};
  return {a.union_slot[list + e], a.union_idx[list + e]};
}

// `last`: the last chunk that a token sees, -1 where there is no token.  The slot of one behind it is not looked at.
__device__ __forceinline__ Entry check_entry(const PagesArgs &a, RawEntry r, bool there, int last, int64_t staged) {
  if (!there) return {0, INT_MAX};
  const int slot = r.slot, idx = r.idx;
  const bool ok = idx >= 0 && idx < a.C && (idx > last || (slot >= 0 ? slot < a.hot_slots : -(int64_t)slot - 1 < staged));
  if (!ok) {
    set_status(a.raised, DD_ERR_DEVICE_CHECK);
    return {0, INT_MAX};
  }
  return {slot, idx << a.cs_log};
}

__device__ __forceinline__ Entry load_entry(const PagesArgs &a, int64_t list, int e, int n, int64_t staged) {
  return check_entry(a, fetch_entry(a, list, e, n), e < n, INT_MAX, staged);
}

__device__ __forceinline__ int64_t staged_slots(const PagesArgs &a) {
  if (!a.miss_count) return a.max_misses;
  const int64_t m = *a.miss_count;
  return m < 0 ? 0 : (m < a.max_misses ? m : a.max_misses);
}

// How many of a list's first n entries (ascending chunks) lie at or before chunk `last`: a
// search by the whole warp, 32 places a look.
__device__ __forceinline__ int entries_up_to(const int32_t *idx, int n, int last, int lane) {
  if (n == 0 || idx[n - 1] <= last) return n;
  int lo = 0, hi = n - 1;                         // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const uint32_t in = __ballot_sync(0xffffffffu, at < hi && idx[at] <= last);
    const int k = __popc(in);                     // entries at lo, lo + step, .. lo + (k - 1) step are in
    if (k == 0) return lo;
    const int l2 = lo + (k - 1) * step + 1;
    hi = min(hi, lo + k * step);
    lo = min(l2, hi);
  }
  return lo;
}

// Half of the columns of a chunk into a tile; a chunk that is not there (position INT_MAX) becomes zeros, as rows
// behind a pool's last read as zeros.
__device__ __forceinline__ void load_chunk(const CUtensorMap &hot, const CUtensorMap &far, const PagesArgs &a, int slot,
                                           int pos, int half, uint32_t dst, uint32_t bar) {
  const bool staged = pos != INT_MAX && slot < 0;
  const int64_t row = pos == INT_MAX ? (a.hot_slots > 0 ? a.hot_slots : 1) : (staged ? -(int64_t)slot - 1 : slot);
  tma_load_2d(dst + half * kTileHalfBytes, staged ? &far : &hot, 64 * half, (int)row << a.cs_log, bar);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)((unsigned)(a + b - 1) / (unsigned)b); }

// A CTA's waits: the first that runs out (2 s) ends the CTA's work, and the others give up with it.
__device__ __forceinline__ bool wait_or_dead(uint32_t bar, uint32_t parity, volatile int *dead, int32_t *raised) {
  if (mbar_try_wait(bar, parity & 1u)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity & 1u)) return true;
    if ((it & 63u) == 0) {
      if (*dead) return false;
      if (globaltimer_ns() - t0 > 2000000000ull) {
        *dead = 1;
        set_status(raised, DD_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// One thread of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
  return r != 0;
}

// A warp's 32 lanes of tensor memory, 32 columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float *v) {
#define DD_U(i) __float_as_uint(v[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(DD_U(0)), "r"(DD_U(1)), "r"(DD_U(2)), "r"(DD_U(3)), "r"(DD_U(4)), "r"(DD_U(5)), "r"(DD_U(6)), "r"(DD_U(7)),
      "r"(DD_U(8)), "r"(DD_U(9)), "r"(DD_U(10)), "r"(DD_U(11)), "r"(DD_U(12)), "r"(DD_U(13)), "r"(DD_U(14)),
      "r"(DD_U(15)), "r"(DD_U(16)), "r"(DD_U(17)), "r"(DD_U(18)), "r"(DD_U(19)), "r"(DD_U(20)), "r"(DD_U(21)),
      "r"(DD_U(22)), "r"(DD_U(23)), "r"(DD_U(24)), "r"(DD_U(25)), "r"(DD_U(26)), "r"(DD_U(27)), "r"(DD_U(28)),
      "r"(DD_U(29)), "r"(DD_U(30)), "r"(DD_U(31))
      : "memory");
#undef DD_U
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Values of a load that has been waited for: nothing that uses them moves in front of this.
__device__ __forceinline__ void tmem_ready(float *v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                    "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                    "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                    "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28])
               :: "memory");
  asm volatile("" : "+f"(v[29]), "+f"(v[30]), "+f"(v[31]) :: "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                          int accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two floats at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// 32 bytes to an address that is a multiple of 32: a thread that writes a row of its own fills a sector each time.
__device__ __forceinline__ void store32(void *to, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The largest of three; a NaN counts as nothing.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The context's counters for these kernels, zero between launches: items handed out,
// CTAs done, then the parts that have arrived of each row tile that is cut.
struct WorkCounters {
  int32_t *ctr;
  int n;          // arrival counters
};

// The launch's last CTA reports its error and leaves the counters as it found them: whoever joins parts clears
// their counter, and where a wait ran out some may never be joined.  All threads, after their
// CTA's last arrival and a barrier.
__device__ __forceinline__ void leave_counters(const WorkCounters &w, const PagesArgs &a, int *last) {
  if (threadIdx.x == 0) {
    int what = 0;                                   // 1: the last one, 2: and there is an error
    __threadfence();
    if (atomicAdd(w.ctr + 1, 1) == (int)gridDim.x - 1) {
      __threadfence();
      const int32_t error = load_status(a.raised);
      what = error != 0 ? 2 : 1;
      if (error != 0) set_status(a.status, error), *a.raised = 0;
    }
    *last = what;
  }
  __syncthreads();
  if (!*last) return;
  if (*last == 2)
    for (int i = threadIdx.x; i < w.n; i += blockDim.x) w.ctr[2 + i] = 0;
  if (threadIdx.x < 2) w.ctr[threadIdx.x] = 0;
}

constexpr int kCtrPerCta = 32;      // arrival counters per CTA of the grid (one CTA an SM)

// host: tensor maps (bf16, 128-byte swizzle), made anew for every call (dd_tmap.cu)
// A pool [slots * cs, 128] (below 2^31 rows), boxes of one slot's rows x 64 columns; rows behind the last read as zeros.
bool make_pages_map(CUtensorMap *map, const void *base, int64_t slots, int cs);
// Query rows [B, T, Hq, 128] with strides in elements, boxes of 64 columns x G heads x tt tokens.
bool make_rows_map(CUtensorMap *map, const void *q, const int64_t *stride, int B, int T, int Hq, int G, int tt);

struct ExtendArgs {
  PagesArgs p;
  const void *q;
  int64_t q_stride[3];
  const void *Khot, *Vhot, *Kst, *Vst;
  void *out;
  int64_t out_stride[3];
  float *lse;
  float *parts;          // extend_workspace() bytes
  int32_t *ctr;          // 2 + kCtrPerCta * sm_count counters, zero (and left zero)
  const void *dummy;     // 16 KB of device memory, the base of a pool without slots
  int sm_count;
};
int64_t extend_workspace(int B, int T, int Hq, int Hkv, int sm_count);
cudaError_t launch_extend(const ExtendArgs &a, cudaStream_t s);

struct WeightsArgs {
  PagesArgs p;
  const void *q;
  int64_t q_stride[3];
  const void *Khot, *Kst;
  const float *lse;
  float *weight;
  int window;
  float decay;
  float *parts;          // weights_workspace() bytes
  int32_t *ctr;
  const void *dummy;
  int sm_count;
};
int64_t weights_workspace(int sm_count);
cudaError_t launch_weights(const WeightsArgs &a, cudaStream_t s);

struct EvictArgs {
  const float *weight;
  const int32_t *kv_len, *new_len, *resident_slot;
  int32_t *resident_out, *slot_chunk, *last_used, *evicted, *evicted_cnt, *list_idx, *list_slot, *list_cnt;
  int units, Hkv, C, cs, S, keep, first, last, step, umax;
  int32_t *status;
  uint32_t *launches, *raised;   // [units] launches so far, the same for all units; [1] the last one with an error
};
cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s);

}  // namespace dd

#endif  // DD_PAGES_CUH_
