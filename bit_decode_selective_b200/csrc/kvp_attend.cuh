// kvp_attend.cuh -- what the attention kernels of the paged 4-bit cache share:
// the call's arguments, a sequence's bounds and the tiles its queries see.
#pragma once

#include <atomic>

#include "kvp.cuh"

namespace sf {

struct KvpAttendArgs {
  const uint8_t* pool;
  const void* q;
  void* out;
  int64_t q_row, q_head;
  const int32_t *cu_q, *pages, *lens;
  int32_t* bad;
  int n_pages, page_shift, h_kv, h_q, group;  // group: query heads per KV head
  int n_q, batch, max_pages, window, sinks;   // window < max_pages * page, 0: none
  uint32_t group_mul, group_shift;            // n / group = n * group_mul >> group_shift, 0 <= n < 2^31
  float scale_log2;                           // scale * log2(e)
  int few_rows;                               // sequences of at most this many rows are the few-row kernel's
  void* ws;
};

// Raises a kernel's dynamic shared memory limit, once per device.
template <auto kernel>
inline cudaError_t kvp_allow_smem(int bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

// Few-row kernel (kvp_decode.cu): rows = queries x group of one sequence and KV head.
size_t kvp_decode_workspace(int d, int rows);
sf_status launch_kvp_decode(const KvpAttendArgs& a, int d, sf_dtype dtype, int rows, cudaStream_t s);

// Many-row kernel (kvp_prefill.cu).
size_t kvp_prefill_workspace(int d);
sf_status launch_kvp_prefill(const KvpAttendArgs& a, int d, sf_dtype dtype, cudaStream_t s);

// The multiplier and shift of a division by d >= 1: with 2^(s-1) < d <= 2^s,
// ceil(2^(31+s) / d) is below 2^32 and exact for numerators below 2^31.
inline void kvp_divisor(uint32_t d, uint32_t& mul, uint32_t& shift) {
  uint32_t s = 0;
  while ((1ull << s) < d) s++;
  mul = (uint32_t)(((1ull << (31 + s)) + d - 1) / d), shift = 31 + s;
}
__device__ __forceinline__ int kvp_by_group(const KvpAttendArgs& a, int n) {
  return (int)((uint64_t)(uint32_t)n * a.group_mul >> a.group_shift);
}

__device__ __forceinline__ void kvp_note_bad(int32_t* bad) {
  if (bad) atomicAdd(bad, 1);
}

// Sequence b: its query rows [q0, q0 + n) and its length, clamped to what the
// call can hold.
struct KvpSeq {
  int q0, n, len;
};
__device__ __forceinline__ KvpSeq kvp_seq(const KvpAttendArgs& a, int b) {
  KvpSeq s;
  if (a.cu_q) {
    const int r0 = a.cu_q[b], r1 = a.cu_q[b + 1];
    s.q0 = min(max(r0, 0), a.n_q);
    const int e = min(max(r1, s.q0), a.n_q);
    if (s.q0 != r0 || e != r1) kvp_note_bad(a.bad);
    s.n = e - s.q0;
  } else {
    s.n = a.n_q / a.batch;
    s.q0 = b * s.n;
  }
  const long cap = (long)a.max_pages << a.page_shift;
  const int l = a.lens[b];
  s.len = l < 0 ? 0 : (int)min((long)l, cap);
  if (s.len != l) kvp_note_bad(a.bad);
  return s;
}

// The 16-token tiles that queries at positions p0 .. p1 see, in order: `sink`
// tiles from the start of the sequence, then those from tile `first` on.  Positions
// before the sequence see nothing and count as -1: p0 - window stays within 32 bits.
struct KvpSpan {
  int p0, p1, sink, first, tiles;
  __device__ __forceinline__ int tile(int i) const { return i < sink ? i : i - sink + first; }
};
__device__ __forceinline__ KvpSpan kvp_span(const KvpAttendArgs& a, int p0, int p1) {
  KvpSpan s;
  p0 = max(p0, -1);
  s.p0 = p0, s.p1 = p1;
  const int lo = a.window ? max(0, p0 - a.window + 1) : 0;
  s.first = lo >> 4;
  s.sink = min((min(a.sinks, lo) + 15) >> 4, s.first);
  s.tiles = p1 < 0 ? 0 : s.sink + (p1 >> 4) + 1 - s.first;
  return s;
}

// ---- the cut of the work ----------------------------------------------------
//
// An item is (sequence, tile of ROWS query rows, KV head); its work is counted
// in steps of STEP cache tiles, after EXTRA steps' worth of time for its queries
// and outputs.  The items lie end to end (sequences, row tiles,
// KV heads, in that order) and the line of steps is cut into equal ranges, one
// per CTA, on the device: the host needs no length.  Parts of an item that
// several CTAs share are joined by a merge kernel in the order of the CTAs.
// FEW: the sequences of at most few_rows rows, else the others.
template <int ROWS, int STEP, int EXTRA, bool FEW>
struct KvpItem {
  static constexpr int kExtra = EXTRA;
  int b, rt, g;
  KvpSeq seq;
  KvpSpan span;
  int steps;

  static __device__ __forceinline__ int row_tiles(const KvpAttendArgs& a, const KvpSeq& s) {
    const long rows = (long)s.n * a.group;
    return rows == 0 || (rows <= a.few_rows) != FEW ? 0 : (int)((rows + ROWS - 1) / ROWS);
  }
  static __device__ __forceinline__ KvpSpan span_of(const KvpAttendArgs& a, const KvpSeq& s, int rt) {
    const int last = min((rt + 1) * ROWS, s.n * a.group) - 1;
    return kvp_span(a, s.len - s.n + kvp_by_group(a, rt * ROWS), s.len - s.n + kvp_by_group(a, last));
  }
  static __device__ __forceinline__ int steps_of(const KvpSpan& s) { return max(1, (s.tiles + STEP - 1) / STEP); }
  // The end of the item that starts at `at`, and the steps of it [s0, s1) that
  // lie in [u0, u1) (none: s0 == s1).
  __device__ __forceinline__ long end(long at) const { return at + EXTRA + steps; }
  __device__ __forceinline__ int2 part(long at, long u0, long u1) const {
    const int s0 = (int)min(max(u0 - at - EXTRA, 0l), (long)steps), s1 = (int)min(max(u1 - at - EXTRA, 0l), (long)steps);
    return make_int2(s0, s1);
  }
  __device__ __forceinline__ void set(const KvpAttendArgs& a) {
    span = span_of(a, seq, rt);
    steps = steps_of(span);
  }
  __device__ __forceinline__ void next(const KvpAttendArgs& a) {
    if (++g < a.h_kv) return;
    g = 0;
    if (++rt >= row_tiles(a, seq)) {
      rt = 0;
      do seq = kvp_seq(a, ++b);
      while (row_tiles(a, seq) == 0);
    }
    set(a);
  }
};

// This CTA's range [u0, u1) of the line (u0 == u1: nothing), and the place `at`
// on the line of the item where it starts.  The first `more` ranges have size
// `each` + 1, the others `each`.  The line is counted in 64 bits, but divided in 32:
// a line of 2^31 steps or more is cut in larger units.
struct KvpRange {
  long u0, u1, at;
  uint32_t each, more;
  int unit;
  __device__ __forceinline__ long begin(uint32_t cta) const {
    return ((long)cta * each + min(cta, more)) << unit;
  }
  // the CTA whose range holds step u of the line
  __device__ __forceinline__ uint32_t cta_of(long u) const {
    const uint32_t x = (uint32_t)(u >> unit), big = more * (each + 1);
    return x < big ? x / (each + 1) : more + (x - big) / each;
  }
};
template <typename Item>
struct KvpRangeShared {
  long scan[32];
  long at;
  Item it;
};
// The KV head whose item holds the step `off` from the first head's start, `each`
// steps an item: off passes 32 bits only with very many heads and tokens.
__device__ __forceinline__ int kvp_head_at(long off, int each) {
  return (int)(off >> 32 ? off / each : (uint32_t)off / (uint32_t)each);
}
// The size of the ranges, and this CTA's.  False: it has none.
__device__ __forceinline__ bool kvp_cut(KvpRange& r, long total, int min_steps) {
  r.u0 = r.u1 = r.at = 0;
  r.unit = 0;
  while (total >> r.unit >> 31) r.unit++;  // at most 2^31 units: nothing below passes 32 bits
  const uint32_t units = (uint32_t)((total + (1l << r.unit) - 1) >> r.unit);
  const uint32_t ctas = min(gridDim.x, (units + min_steps - 1) / min_steps);
  if (blockIdx.x >= ctas) return false;
  r.each = units / ctas, r.more = units - r.each * ctas;
  r.u0 = r.begin(blockIdx.x), r.u1 = min(r.begin(blockIdx.x + 1), total);
  if (r.u0 < total) return true;
  r.u1 = r.u0;  // (the last unit can be a short one)
  return false;
}
__device__ __forceinline__ long kvp_scan(long x) {  // inclusive sum over the lanes
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// kvp_range for batches of at most 32 * kKvpFew sequences with few row tiles:
// every warp finds the place by itself, without a barrier (0.3 us of a call with
// one sequence of 8192 tokens).
constexpr int kKvpFew = 2;
template <typename Item>
__device__ __forceinline__ KvpRange kvp_range_few(const KvpAttendArgs& a, int min_steps, Item& it) {
  const int lane = threadIdx.x & 31;
  KvpSeq seq[kKvpFew];
  long steps[kKvpFew], mine = 0;
#pragma unroll
  for (int k = 0; k < kKvpFew; k++) {
    const int b = lane * kKvpFew + k;
    seq[k].q0 = seq[k].n = seq[k].len = 0;
    if (b < a.batch) seq[k] = kvp_seq(a, b);
    steps[k] = 0;
    const int n = Item::row_tiles(a, seq[k]);
    for (int rt = 0; rt < n; rt++) steps[k] += Item::kExtra + Item::steps_of(Item::span_of(a, seq[k], rt));
    steps[k] *= a.h_kv;
    mine += steps[k];
  }
  const long upto = kvp_scan(mine);
  KvpRange r;
  if (!kvp_cut(r, __shfl_sync(0xffffffffu, upto, 31), min_steps)) return r;
  // the lane whose sequences hold u0 finds the item
  int b = 0, rt = 0, g = 0;
  KvpSeq s = seq[0];
  long at = upto - mine;
  const bool here = r.u0 >= at && r.u0 < upto;
  if (here) {
#pragma unroll
    for (int k = 0; k < kKvpFew - 1; k++)
      if (b == k && r.u0 >= at + steps[k]) at += steps[k], b = k + 1, s = seq[k + 1];
    for (;; rt++) {
      const int st = Item::kExtra + Item::steps_of(Item::span_of(a, s, rt));
      const long all = (long)st * a.h_kv;
      if (r.u0 < at + all) {
        g = kvp_head_at(r.u0 - at, st);
        at += (long)g * st;
        break;
      }
      at += all;
    }
    b += lane * kKvpFew;
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  it.b = __shfl_sync(0xffffffffu, b, from), it.rt = __shfl_sync(0xffffffffu, rt, from);
  it.g = __shfl_sync(0xffffffffu, g, from), r.at = __shfl_sync(0xffffffffu, at, from);
  it.seq.q0 = __shfl_sync(0xffffffffu, s.q0, from), it.seq.n = __shfl_sync(0xffffffffu, s.n, from);
  it.seq.len = __shfl_sync(0xffffffffu, s.len, from);
  it.set(a);
  return r;
}

// All threads of the CTA call it, the work of the sequences split over them:
// thread by thread, or with SPREAD warp by warp, the lanes over the row tiles of
// long queries.  `it` is set where the range is not empty.
template <int THREADS, bool SPREAD, typename Item>
__device__ __forceinline__ KvpRange kvp_range(const KvpAttendArgs& a, int min_steps, KvpRangeShared<Item>& sh, Item& it) {
  if (!SPREAD && a.batch <= 32 * kKvpFew) return kvp_range_few(a, min_steps, it);
  constexpr int kParts = SPREAD ? THREADS / 32 : THREADS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int me = SPREAD ? warp : tid;
  const int per = (a.batch + kParts - 1) / kParts;
  const int b0 = min(me * per, a.batch), b1 = min(b0 + per, a.batch);
  // steps of my sequences' items; SPREAD: of my lane's row tiles
  long mine = 0;
  for (int b = b0; b < b1; b++) {
    const KvpSeq s = kvp_seq(a, b);
    const int n = Item::row_tiles(a, s);
    for (int rt = SPREAD ? lane : 0; rt < n; rt += SPREAD ? 32 : 1) mine += Item::kExtra + Item::steps_of(Item::span_of(a, s, rt));
  }
  mine *= a.h_kv;
  const long upto = kvp_scan(mine);
  if (lane == 31) sh.scan[warp] = upto;
  __syncthreads();
  long before = 0, total = 0;  // of the warps before this one, of all
#pragma unroll
  for (int w = 0; w < THREADS / 32; w++) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  KvpRange r;
  if (!kvp_cut(r, total, min_steps)) return r;  // all threads alike
  // the part that holds u0 finds its item
  const long from = SPREAD ? before : before + upto - mine, to = SPREAD ? before + sh.scan[warp] : before + upto;
  if (r.u0 >= from && r.u0 < to) {
    long at = from;
    bool found = false;
    for (int b = b0; b < b1 && !found; b++) {
      const KvpSeq s = kvp_seq(a, b);
      const int n = Item::row_tiles(a, s);
      for (int rt0 = 0; rt0 < n && !found; rt0 += SPREAD ? 32 : 1) {
        const int rt = rt0 + (SPREAD ? lane : 0);
        const int st = rt < n ? Item::kExtra + Item::steps_of(Item::span_of(a, s, rt)) : 0;
        const long all = (long)st * a.h_kv;
        const long end = SPREAD ? kvp_scan(all) : all;  // inclusive sum over the row tiles at hand
        const bool here = r.u0 >= at + end - all && r.u0 < at + end;
        if (here) {
          const int g = kvp_head_at(r.u0 - (at + end - all), st);
          sh.it.b = b, sh.it.rt = rt, sh.it.g = g;
          sh.it.seq = s;
          sh.it.set(a);
          sh.at = at + end - all + (long)g * st;
        }
        if (SPREAD) {
          found = __any_sync(0xffffffffu, here);
          at += __shfl_sync(0xffffffffu, end, 31);
        } else {
          found = here;
          at += end;
        }
      }
    }
  }
  __syncthreads();
  it = sh.it;
  r.at = sh.at;
  return r;
}

// An item that several CTAs share, written by the one with its first step.
struct KvpShared {
  int q_row, row0, rows, head0;  // first query row of the sequence, first row, rows, first query head
  int parts, cta, pad[2];       // CTAs that share it, the first of them
};
// How many CTAs share the item that ends at `end` and has its first step in
// this one's range.
__device__ __forceinline__ int kvp_sharers(const KvpRange& r, long end) {
  return (int)(r.cta_of(end - 1) - blockIdx.x + 1);
}

__device__ __forceinline__ bool kvp_sees(const KvpAttendArgs& a, int p, int j) {
  return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}
// Whether every query at p0 .. p1 sees all of the `count` tokens from j on.
__device__ __forceinline__ bool kvp_sees_all(const KvpAttendArgs& a, int p0, int p1, int j, int count) {
  return j + count - 1 <= p0 && (a.window == 0 || j > p1 - a.window || j + count <= a.sinks);
}
// Whether some query at p0 .. p1 sees token j (p0 .. p1 without gaps).
__device__ __forceinline__ bool kvp_some_sees(const KvpAttendArgs& a, int p0, int p1, int j) {
  return j <= p1 && (a.window == 0 || j > p0 - a.window || j < a.sinks);
}

}  // namespace sf
