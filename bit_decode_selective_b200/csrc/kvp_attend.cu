// kvp_attend.cu -- attention over the paged 4-bit KV cache (include/sf.h,
// sf_kvp_attend): ragged causal queries, a sliding window and sinks.
#include <climits>
#include <cmath>

#include "kvp_attend.cuh"

namespace sf {
namespace {

// Sequences of at most this many rows (queries x query heads per KV head) go to
// the few-row kernel.
constexpr int kFewRows = 64;

// Rows that a sequence of the few-row kernel is expected to have: the average.
int few_rows(int n_q, int batch, int group) {
  const long long rows = ((long long)n_q + batch - 1) / batch * group;
  return rows < kFewRows ? (int)rows : kFewRows;
}

// One warp per (query, head), a token per lane and step for the logits, D / 32
// elements per lane for the output.
template <typename T, int D>
__global__ void __launch_bounds__(128) kvp_attend_plain_kernel(KvpAttendArgs a) {
  using L = KvpTile<D>;
  constexpr int E = D / 32;
  __shared__ float qs[4][D];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z;
  const KvpSeq seq = kvp_seq(a, b);
  const int q0 = seq.q0, n = seq.n, len = seq.len;
  if ((long)n * a.group <= a.few_rows) return;
  const long unit = (long)blockIdx.x * 4 + warp;
  const int i = (int)(unit / a.h_q), h = (int)(unit % a.h_q), g = h / a.group;
  if (i >= n) return;
  const int p = len - n + i;
  const T* qr = static_cast<const T*>(a.q) + (q0 + i) * a.q_row + h * a.q_head;
  for (int e = lane; e < D; e += 32) qs[warp][e] = Elem<T>::to_float(qr[e]) * a.scale_log2;
  __syncwarp();
  float mx = -INFINITY, sum = 0.f, acc[E] = {};
  const int lo = a.window ? max(0, p - a.window + 1) : 0;
  const int n_sink = min(a.sinks, lo);
  const int total = p < 0 ? 0 : n_sink + (p + 1 - lo);
  for (int c0 = 0; c0 < total; c0 += 32) {
    const int idx = c0 + lane;
    const int j = idx < n_sink ? idx : idx - n_sink + lo;
    float x = -INFINITY;
    long tile_at = -1;
    if (idx < total) {
      const int page = a.pages[(long)b * a.max_pages + (j >> a.page_shift)];
      if (page >= 0 && page < a.n_pages) {
        const int in_page = j & ((1 << a.page_shift) - 1);
        tile_at = (((long)page * a.h_kv + g << (a.page_shift - 4)) + (in_page >> 4)) * L::kBytes;
        const uint8_t* tile = a.pool + tile_at;
        const int t = j & 15;
        x = 0.f;
        for (int grp = 0; grp < L::G; grp++) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(tile + L::kKeyCodes + (grp * 16 + t) * 16);
          const uint32_t z = *reinterpret_cast<const uint32_t*>(tile + L::kKeyGrid + (t * L::G + grp) * 4);
          const float s = h2f((uint16_t)(z & 0xffff)), m = h2f((uint16_t)(z >> 16));
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int e = 0; e < 32; e++)
            x = fmaf(qs[warp][grp * 32 + e], fmaf((float)((w[e >> 3] >> (4 * (e & 7))) & 15u), s, m), x);
        }
      } else {
        kvp_note_bad(a.bad);
      }
    }
    float top = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float now = fmaxf(mx, top);
    if (now == -INFINITY) continue;  // the same in every lane
    const float w = exp2f(x - now), old = exp2f(mx - now);
    mx = now;
    sum = sum * old + w;
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] *= old;
    for (int l = 0; l < 32; l++) {
      const float wl = __shfl_sync(0xffffffffu, w, l);
      const long at = __shfl_sync(0xffffffffu, tile_at, l);
      const int t = __shfl_sync(0xffffffffu, j, l) & 15;
      if (at < 0) continue;
      const uint8_t* tile = a.pool + at;
      const int e0 = lane * E, grp = e0 >> 5;
      const uint16_t* vz =
          reinterpret_cast<const uint16_t*>(tile + L::kValueGrid) + ((t >> 1) * L::G + grp) * 4 + (t & 1);
      const float s = h2f(vz[0]), m = h2f(vz[2]);
#pragma unroll
      for (int e = 0; e < E; e++) {
        const int d = (e0 + e) & 31;
        const uint32_t c = (tile[L::kValueCodes + (grp * 16 + t) * 16 + (d >> 1)] >> (4 * (d & 1))) & 15u;
        acc[e] = fmaf(wl, fmaf((float)c, s, m), acc[e]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  T* o = static_cast<T*>(a.out) + ((long)(q0 + i) * a.h_q + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e++) o[e] = Elem<T>::from_float(acc[e] * inv);
}

template <typename T, int D>
sf_status launch_attend(const KvpAttendArgs& a, cudaStream_t s) {
  const long units = (long)(a.cu_q ? a.n_q : a.n_q / a.batch) * a.h_q;
  SF_CUDA(launch_pdl(kvp_attend_plain_kernel<T, D>, dim3((unsigned)((units + 3) / 4), 1, a.batch), dim3(128), 0, s, a));
  return SF_OK;
}

sf_status check_attend(const sf_kvp* kv, int n_q, int batch, int h_q) {
  const sf_status st = check_kvp(kv);
  if (st != SF_OK) return st;
  SF_REQUIRE(batch > 0 && n_q >= 0, "bad attention shape: batch=%d n_q=%d", batch, n_q);
  SF_UNSUPPORTED(batch <= 65535, "batch=%d above 65535", batch);
  SF_REQUIRE(h_q > 0 && h_q % kv->h_kv == 0, "h_q=%d must be a positive multiple of h_kv=%d", h_q, kv->h_kv);
  SF_UNSUPPORTED((long long)n_q * h_q <= INT_MAX / 2, "n_q=%d x h_q=%d is too large", n_q, h_q);
  return SF_OK;
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" size_t sf_kvp_attend_workspace_bytes(const sf_kvp* kv, int n_q, int batch, int h_q) {
  if (check_attend(kv, n_q, batch, h_q) != SF_OK || n_q == 0) return 0;
  return kvp_decode_workspace(kv->d, few_rows(n_q, batch, h_q / kv->h_kv));
}

extern "C" sf_status sf_kvp_attend(const sf_kvp* kv, const void* q, int64_t q_row, int64_t q_head, sf_dtype dtype,
                                   int n_q, const int32_t* cu_q, const int32_t* pages, int max_pages,
                                   const int32_t* lens, int batch, int h_q, float scale, int window, int sinks,
                                   void* out, int32_t* bad, void* ws, size_t ws_bytes, sf_stream_t stream) {
  const sf_status st = check_attend(kv, n_q, batch, h_q);
  if (st != SF_OK) return st;
  SF_REQUIRE(dtype == SF_F16 || dtype == SF_BF16 || dtype == SF_F32, "dtype %d unknown", (int)dtype);
  SF_UNSUPPORTED(dtype != SF_F32, "queries are fp16 or bf16");
  SF_REQUIRE(std::isfinite(scale), "scale must be finite");
  SF_REQUIRE(window >= 0 && sinks >= 0, "window=%d and sinks=%d must not be negative", window, sinks);
  SF_REQUIRE(max_pages > 0, "max_pages=%d < 1", max_pages);
  SF_UNSUPPORTED((long long)max_pages * kv->page <= INT_MAX, "%d pages of %d tokens per sequence pass 2^31",
                 max_pages, kv->page);
  SF_REQUIRE(pages && lens && (((uintptr_t)pages | (uintptr_t)lens | (uintptr_t)cu_q | (uintptr_t)bad) & 3) == 0,
             "pages and lens must be non-null; index arrays 4-byte aligned");
  SF_REQUIRE(cu_q || n_q % batch == 0, "n_q=%d is not a multiple of batch=%d, and there is no cu_q", n_q, batch);
  if (n_q == 0) return SF_OK;
  SF_REQUIRE(q && aligned16(q) && out && aligned16(out), "q and out must be non-null 16-byte aligned device pointers");
  SF_REQUIRE(q_row >= 0 && q_head >= 0 && q_row % 8 == 0 && q_head % 8 == 0,
             "q strides (%lld, %lld) must be whole multiples of 16 bytes", (long long)q_row, (long long)q_head);
  const size_t need = sf_kvp_attend_workspace_bytes(kv, n_q, batch, h_q);
  if (!ws || ws_bytes < need) {
    set_error("workspace: need %zu bytes, got %zu", need, ws ? ws_bytes : (size_t)0);
    return SF_ERR_WORKSPACE;
  }
  SF_REQUIRE(aligned16(ws), "ws must be 16-byte aligned");
  KvpAttendArgs a = {};
  a.pool = (const uint8_t*)kv->pool, a.q = q, a.out = out, a.q_row = q_row, a.q_head = q_head;
  a.cu_q = cu_q, a.pages = pages, a.lens = lens, a.bad = bad;
  a.n_pages = kv->n_pages, a.h_kv = kv->h_kv, a.h_q = h_q, a.group = h_q / kv->h_kv;
  while ((1 << a.page_shift) < kv->page) a.page_shift++;
  a.n_q = n_q, a.batch = batch, a.max_pages = max_pages, a.sinks = sinks;
  a.window = window < (long long)max_pages * kv->page ? window : 0;  // as wide as any sequence: no window
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.few_rows = kFewRows;
  a.ws = ws;
  cudaStream_t s = as_stream(stream);
  // without cu_q every sequence has the same number of rows; with it the
  // kernels take the sequences that are theirs
  const long long each = (long long)(n_q / batch) * a.group;
  if (cu_q || each <= kFewRows) {
    const sf_status e = launch_kvp_decode(a, kv->d, dtype, few_rows(n_q, batch, a.group), s);
    if (e != SF_OK) return e;
  }
  if (cu_q ? (long long)n_q * a.group <= kFewRows : each <= kFewRows) return SF_OK;
  if (kv->d == 128)
    return dtype == SF_F16 ? launch_attend<__half, 128>(a, s) : launch_attend<__nv_bfloat16, 128>(a, s);
  return dtype == SF_F16 ? launch_attend<__half, 64>(a, s) : launch_attend<__nv_bfloat16, 64>(a, s);
}
