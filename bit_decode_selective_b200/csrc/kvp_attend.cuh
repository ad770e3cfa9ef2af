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
// tiles from the start of the sequence, then those from tile `first` on.
struct KvpSpan {
  int p0, p1, sink, first, tiles;
  __device__ __forceinline__ int tile(int i) const { return i < sink ? i : i - sink + first; }
};
__device__ __forceinline__ KvpSpan kvp_span(const KvpAttendArgs& a, int p0, int p1) {
  KvpSpan s;
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
    return kvp_span(a, s.len - s.n + rt * ROWS / a.group, s.len - s.n + last / a.group);
  }
  static __device__ __forceinline__ int steps_of(const KvpSpan& s) { return max(1, (s.tiles + STEP - 1) / STEP); }
  // Steps of one sequence, over its row tiles (not yet times the KV heads).
  static __device__ __forceinline__ long seq_steps(const KvpAttendArgs& a, const KvpSeq& s) {
    const int n = row_tiles(a, s);
    long sum = 0;
    for (int rt = 0; rt < n; rt++) sum += EXTRA + steps_of(span_of(a, s, rt));
    return sum;
  }
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

// This CTA's range [u0, u1) of the line (u0 == u1: nothing), and the item and
// place `at` on the line where it starts.  All threads call it.
struct KvpRange {
  long u0, u1, at, total, ctas;
};
struct KvpRangeShared {
  long scan[32];
  long at;
  int b, rt, g;
};
template <int THREADS, typename Item>
__device__ __forceinline__ KvpRange kvp_range(const KvpAttendArgs& a, int min_steps, KvpRangeShared& sh, Item& it) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long mine = 0;
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  for (int b = b0; b < b1; b++) mine += Item::seq_steps(a, kvp_seq(a, b)) * a.h_kv;
  long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.scan[warp] = upto;
  __syncthreads();
  KvpRange r;
  r.total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; w++) {
    if (w < warp) upto += sh.scan[w];
    r.total += sh.scan[w];
  }
  r.ctas = min((long)gridDim.x, (r.total + min_steps - 1) / min_steps);
  r.u0 = r.u1 = 0;
  if ((long)blockIdx.x >= r.ctas) return r;  // all threads alike
  r.u0 = r.total * blockIdx.x / r.ctas, r.u1 = r.total * (blockIdx.x + 1) / r.ctas;
  if (r.u0 >= upto - mine && r.u0 < upto) {  // one thread
    long at = upto - mine;
    bool found = false;
    for (int b = b0; b < b1 && !found; b++) {
      const KvpSeq s = kvp_seq(a, b);
      const int n = Item::row_tiles(a, s);
      for (int rt = 0; rt < n && !found; rt++) {
        const int st = Item::kExtra + Item::steps_of(Item::span_of(a, s, rt));
        if (r.u0 < at + (long)st * a.h_kv) {
          sh.b = b, sh.rt = rt, sh.g = (int)((r.u0 - at) / st);
          sh.at = at + (long)sh.g * st;
          found = true;
        } else {
          at += (long)st * a.h_kv;
        }
      }
    }
  }
  __syncthreads();
  it.b = sh.b, it.rt = sh.rt, it.g = sh.g;
  it.seq = kvp_seq(a, it.b);
  it.set(a);
  r.at = sh.at;
  return r;
}

// An item that several CTAs share, written by the one with its first step.
struct KvpShared {
  int q_row, row0, rows, head0;  // first query row of the sequence, first row, rows, first query head
  int parts, pad[3];
};
// How many CTAs share the item that ends at `end` and has its first step in
// this one's range.
__device__ __forceinline__ int kvp_sharers(const KvpRange& r, long end) {
  long last = (end * r.ctas + r.total - 1) / r.total - 1;
  while (r.total * (last + 1) / r.ctas < end) last++;
  while (r.total * last / r.ctas >= end) last--;
  return (int)(last - blockIdx.x + 1);
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
