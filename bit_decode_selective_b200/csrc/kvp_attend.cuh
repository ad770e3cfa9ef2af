// kvp_attend.cuh -- what the attention kernels of the paged 4-bit cache share:
// the call's arguments, a sequence's bounds and the tiles its queries see.
#pragma once

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

// Few-row kernel (kvp_decode.cu): rows = queries x group of one sequence and KV head.
size_t kvp_decode_workspace(int d, int rows);
sf_status launch_kvp_decode(const KvpAttendArgs& a, int d, sf_dtype dtype, int rows, cudaStream_t s);

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
