// kvp_cache.cu -- the paged 4-bit KV cache: quantising tokens as they are
// written, and reading them back.
//
// Per group of 32 values w of one token and head: s = fp16((max - min) / 15),
// m = fp16(min), q = clamp(floor((w - m) / s + 1/2), 0, 15), value m + s q
// (include/sf.h).  The decisions are those of fp64 arithmetic with one rounding
// per operation (quant.cuh).
//
// Four neighbouring lanes hold a group, 8 elements each (one 16-byte load of a
// 16-bit type, two of fp32): min and max take two shuffles, and a lane's 8
// codes are one 32-bit word of the tile.
#include <climits>

#include "kvp.cuh"
#include "quant.cuh"

namespace sf {

sf_status check_kvp(const sf_kvp* kv) {
  SF_REQUIRE(kv != nullptr, "null sf_kvp");
  SF_REQUIRE(kv->n_pages > 0 && kv->h_kv > 0, "bad paged cache: n_pages=%d h_kv=%d", kv->n_pages, kv->h_kv);
  SF_UNSUPPORTED(kv->d == 64 || kv->d == 128, "a paged cache has d 64 or 128 (got %d)", kv->d);
  SF_UNSUPPORTED(kv->page >= 16 && kv->page <= 1024 && (kv->page & (kv->page - 1)) == 0,
                 "page=%d is not a power of two in [16, 1024]", kv->page);
  SF_UNSUPPORTED((long long)kv->n_pages * kv->page <= INT_MAX, "%d pages of %d tokens pass 2^31 slots", kv->n_pages,
                 kv->page);
  SF_REQUIRE(kv->pool && aligned16(kv->pool), "pool must be a non-null 16-byte aligned device pointer");
  return SF_OK;
}

namespace {

constexpr int kThreads = 256;

struct CacheArgs {
  uint8_t* pool;
  const void* x[2];  // keys, values (write: inputs; either may be null)
  void* y[2];        // read: outputs
  int64_t row[2], head[2];
  const int32_t* slots;
  int32_t* bad;
  int n, h_kv, page_shift, n_slots;
  int kind0;  // blockIdx.y = 0 handles kind kind0 (0 keys, 1 values)
};

// Byte offset of the tile that holds `slot` for head h.
template <int D>
__device__ __forceinline__ size_t tile_offset(int slot, int h, int h_kv, int page_shift) {
  const int page = slot >> page_shift, in_page = slot & ((1 << page_shift) - 1);
  return (((size_t)page * h_kv + h << (page_shift - 4)) + (in_page >> 4)) * KvpTile<D>::kBytes;
}

__device__ __forceinline__ float tame(float x) {
  x = fminf(fmaxf(x, -kKvpLimit), kKvpLimit);
  return x;
}

template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 f = Elem<T>::to_float2(w[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 a;
    a.x = Elem<T>::from_float2(v[0], v[1]), a.y = Elem<T>::from_float2(v[2], v[3]);
    a.z = Elem<T>::from_float2(v[4], v[5]), a.w = Elem<T>::from_float2(v[6], v[7]);
    *reinterpret_cast<uint4*>(static_cast<T*>(base) + at) = a;
  }
}

// One thread: 8 elements of one (token, head); D / 8 threads a row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kvp_write_kernel(CacheArgs a) {
  using L = KvpTile<D>;
  pdl_trigger();
  pdl_wait();
  const int kind = a.kind0 + blockIdx.y;
  const long unit = (long)blockIdx.x * kThreads + threadIdx.x;
  const long row = unit / (D / 8);
  const int part = (int)(unit % (D / 8));  // 8-element part of the row
  const long tok = row / a.h_kv;
  const int h = (int)(row % a.h_kv);
  const bool in = tok < a.n;
  const int slot = in ? a.slots[tok] : -1;
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (in && !ok && slot != -1 && a.bad && blockIdx.y == 0 && h == 0 && part == 0) atomicAdd(a.bad, 1);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = 0.f;
  if (ok) load8<T>(a.x[kind], tok * a.row[kind] + h * a.head[kind] + part * 8, v);
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = isnan(v[i]) ? 0.f : tame(v[i]);
    lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!ok) return;
  const Grid16 g = group_grid((double)lo, (double)hi, 4);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) word |= (uint32_t)nested_code((double)v[i], g, 0, 15) << (4 * i);
  uint8_t* tile = a.pool + tile_offset<D>(slot, h, a.h_kv, a.page_shift);
  const int grp = part >> 2, t = slot & 15;
  *reinterpret_cast<uint32_t*>(tile + (kind ? L::kValueCodes : L::kKeyCodes) + (grp * 16 + t) * 16 + (part & 3) * 4) =
      word;
  if ((part & 3) == 0) {
    if (kind) {
      uint16_t* vz = reinterpret_cast<uint16_t*>(tile + L::kValueGrid) + ((t >> 1) * L::G + grp) * 4 + (t & 1);
      vz[0] = g.s16, vz[2] = g.m16;
    } else {
      *reinterpret_cast<uint32_t*>(tile + L::kKeyGrid + (t * L::G + grp) * 4) =
          (uint32_t)g.s16 | ((uint32_t)g.m16 << 16);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kvp_read_kernel(CacheArgs a) {
  using L = KvpTile<D>;
  pdl_trigger();
  pdl_wait();
  const int kind = a.kind0 + blockIdx.y;
  const long unit = (long)blockIdx.x * kThreads + threadIdx.x;
  const long row = unit / (D / 8);
  const int part = (int)(unit % (D / 8));
  const long tok = row / a.h_kv;
  const int h = (int)(row % a.h_kv);
  if (tok >= a.n) return;
  const int slot = a.slots[tok];
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (!ok && slot != -1 && a.bad && blockIdx.y == 0 && h == 0 && part == 0) atomicAdd(a.bad, 1);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = 0.f;
  if (ok) {
    const uint8_t* tile = a.pool + tile_offset<D>(slot, h, a.h_kv, a.page_shift);
    const int grp = part >> 2, t = slot & 15;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(tile + (kind ? L::kValueCodes : L::kKeyCodes) +
                                                             (grp * 16 + t) * 16 + (part & 3) * 4);
    float s, m;
    if (kind) {
      const uint16_t* vz =
          reinterpret_cast<const uint16_t*>(tile + L::kValueGrid) + ((t >> 1) * L::G + grp) * 4 + (t & 1);
      s = h2f(vz[0]), m = h2f(vz[2]);
    } else {
      const uint32_t z = *reinterpret_cast<const uint32_t*>(tile + L::kKeyGrid + (t * L::G + grp) * 4);
      s = h2f((uint16_t)(z & 0xffff)), m = h2f((uint16_t)(z >> 16));
    }
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = fmaf((float)((word >> (4 * i)) & 15u), s, m);
  }
  store8<T>(a.y[kind], row * D + part * 8, v);
}

template <typename T>
sf_status launch_cache(const CacheArgs& a, int d, int kinds, bool read, cudaStream_t s) {
  const long units = (long)a.n * a.h_kv * (d / 8);
  const dim3 grid((unsigned)((units + kThreads - 1) / kThreads), kinds);
  if (d == 128)
    SF_CUDA(launch_pdl(read ? kvp_read_kernel<T, 128> : kvp_write_kernel<T, 128>, grid, dim3(kThreads), 0, s, a));
  else
    SF_CUDA(launch_pdl(read ? kvp_read_kernel<T, 64> : kvp_write_kernel<T, 64>, grid, dim3(kThreads), 0, s, a));
  return SF_OK;
}

sf_status launch_cache_any(const CacheArgs& a, int d, int kinds, bool read, sf_dtype dtype, cudaStream_t s) {
  if (dtype == SF_F16) return launch_cache<__half>(a, d, kinds, read, s);
  if (dtype == SF_BF16) return launch_cache<__nv_bfloat16>(a, d, kinds, read, s);
  return launch_cache<float>(a, d, kinds, read, s);
}

CacheArgs cache_args(const sf_kvp* kv, const int32_t* slots, int n, int32_t* bad) {
  CacheArgs a = {};
  a.pool = (uint8_t*)kv->pool;
  a.slots = slots, a.bad = bad, a.n = n, a.h_kv = kv->h_kv;
  a.n_slots = kv->n_pages * kv->page;
  while ((1 << a.page_shift) < kv->page) a.page_shift++;
  return a;
}

sf_status check_rows(const char* name, const void* p, int64_t row, int64_t head, int esz) {
  SF_REQUIRE(aligned16(p), "%s must be 16-byte aligned", name);
  SF_REQUIRE(row >= 0 && head >= 0 && row * esz % 16 == 0 && head * esz % 16 == 0,
             "%s strides (%lld, %lld) must be whole multiples of 16 bytes", name, (long long)row, (long long)head);
  return SF_OK;
}

sf_status check_slots(const sf_kvp* kv, const int32_t* slots, int n, sf_dtype dtype, const int32_t* bad) {
  const sf_status st = check_kvp(kv);
  if (st != SF_OK) return st;
  SF_REQUIRE(dtype == SF_F16 || dtype == SF_BF16 || dtype == SF_F32, "dtype %d unknown", (int)dtype);
  SF_REQUIRE(n >= 0, "n=%d < 0", n);
  SF_REQUIRE(n == 0 || (slots && ((uintptr_t)slots & 3) == 0), "slots must be a non-null 4-byte aligned device pointer");
  SF_REQUIRE(((uintptr_t)bad & 3) == 0, "bad must be 4-byte aligned");
  SF_UNSUPPORTED((long long)n * kv->h_kv * (kv->d / 8) <= (long long)INT_MAX * kThreads, "n=%d is too large", n);
  return SF_OK;
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" sf_status sf_kvp_bytes(int n_pages, int page, int h_kv, int d, size_t* bytes) {
  sf_kvp kv = {n_pages, page, h_kv, d, (void*)16};
  const sf_status st = check_kvp(&kv);
  if (st != SF_OK) return st;
  SF_REQUIRE(bytes, "bytes must be non-null");
  *bytes = (size_t)n_pages * h_kv * (page / 16) * 20 * d;
  return SF_OK;
}

extern "C" sf_status sf_kvp_write(const sf_kvp* kv, const void* k, int64_t k_row, int64_t k_head, const void* v,
                                  int64_t v_row, int64_t v_head, sf_dtype dtype, int n, const int32_t* slots,
                                  int32_t* bad, sf_stream_t stream) {
  sf_status st = check_slots(kv, slots, n, dtype, bad);
  if (st != SF_OK) return st;
  const int esz = dtype == SF_F32 ? 4 : 2;
  if (k && (st = check_rows("k", k, k_row, k_head, esz)) != SF_OK) return st;
  if (v && (st = check_rows("v", v, v_row, v_head, esz)) != SF_OK) return st;
  if (n == 0 || (!k && !v)) return SF_OK;
  CacheArgs a = cache_args(kv, slots, n, bad);
  a.x[0] = k, a.row[0] = k_row, a.head[0] = k_head;
  a.x[1] = v, a.row[1] = v_row, a.head[1] = v_head;
  a.kind0 = k ? 0 : 1;
  return launch_cache_any(a, kv->d, (k ? 1 : 0) + (v ? 1 : 0), false, dtype, as_stream(stream));
}

extern "C" sf_status sf_kvp_read(const sf_kvp* kv, const int32_t* slots, int n, void* k, void* v, sf_dtype dtype,
                                 int32_t* bad, sf_stream_t stream) {
  sf_status st = check_slots(kv, slots, n, dtype, bad);
  if (st != SF_OK) return st;
  SF_REQUIRE((!k || aligned16(k)) && (!v || aligned16(v)), "k and v must be 16-byte aligned");
  if (n == 0 || (!k && !v)) return SF_OK;
  CacheArgs a = cache_args(kv, slots, n, bad);
  a.y[0] = k, a.y[1] = v;
  a.kind0 = k ? 0 : 1;
  return launch_cache_any(a, kv->d, (k ? 1 : 0) + (v ? 1 : 0), true, dtype, as_stream(stream));
}
