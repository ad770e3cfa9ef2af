// kvp_attend.cu -- attention over the paged 4-bit KV cache (include/sf.h,
// sf_kvp_attend): ragged causal queries, a sliding window and sinks.
#include <climits>
#include <cmath>

#include "kvp_attend.cuh"

namespace sf {
namespace {

// Sequences of at most this many rows (queries x query heads per KV head) go to
// the few-row kernel, whose logits are sums of exact products.  Both kernels, in us
// (few rows | many rows; bf16, 8 KV heads, d = 128):
//   rows          16           32           40           48           64
//   1 x 1,024     10 |  16     14 |  16     14 |  16     14 |  17     16 |  17
//   16 x 1,024    19 |  30     32 |  31     37 |  32     38 |  32     51 |  32
//   64 x 1,024    46 |  95     81 |  95     98 |  95    101 |  95    135 |  95
//   1 x 16,384    15 |  34     23 |  35     30 |  36     30 |  36     37 |  36
//   16 x 16,384  101 | 231    176 | 232    250 | 232    252 | 232    331 | 235
//   64 x 16,384  362 | 875    634 | 879    934 | 879    937 | 880   1233 | 883
// So up to 32 rows it is the faster one but for a tie; from there to the limit it is
// kept for its precision, at up to 1.6 times the other's time for batches of 64 rows each.
constexpr int kFewRows = 64;

// The rows by which the few-row kernel's columns are chosen: the average over the
// call's sequences, all that the host knows.  Long sequences beside single tokens
// raise it, many single tokens beside a draft lower it; either costs time only.
int few_rows(int n_q, int batch, int group) {
  const long long rows = ((long long)n_q + batch - 1) / batch * group;
  return rows < kFewRows ? (int)rows : kFewRows;
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
  // the two kernels of a call run one after the other and share the space
  const int group = h_q / kv->h_kv;
  const size_t few = kvp_decode_workspace(kv->d, few_rows(n_q, batch, group));
  if ((long long)n_q * group <= kFewRows) return few;
  const size_t many = kvp_prefill_workspace(kv->d);
  return few > many ? few : many;
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
  kvp_divisor((uint32_t)a.group, a.group_mul, a.group_shift);
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
  return launch_kvp_prefill(a, kv->d, dtype, s);
}
