// kvp_cache.cu -- the paged 4-bit KV cache: quantising tokens as they are
// written, and reading them back.
//
// Per group of 32 values w of one token and head: s = fp16((max - min) / 15),
// m = fp16(min), q = clamp(floor((w - m) / s + 1/2), 0, 15), value m + s q
// (include/sf.h).  The decisions are those of fp64 arithmetic with one rounding
// per operation (quant.cuh).
//
// A thread takes one token of one head, and of every group the quarter that its
// place c among four neighbouring lanes names: 8 elements, one 16-byte load or
// store of a 16-bit type, one 32-bit word of codes.  The eight tokens of a warp
// then touch whole sectors on both sides: 64 bytes of a row, and 128 bytes of a
// tile's codes where their slots follow each other.
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
  SF_UNSUPPORTED(kv->h_kv <= 65535, "h_kv=%d above 65535", kv->h_kv);
  SF_UNSUPPORTED((long long)kv->n_pages * kv->page <= INT_MAX, "%d pages of %d tokens pass 2^31 slots", kv->n_pages,
                 kv->page);
  SF_REQUIRE(kv->pool && aligned16(kv->pool), "pool must be a non-null 16-byte aligned device pointer");
  return SF_OK;
}

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 4;  // per CTA

struct CacheArgs {
  uint8_t* pool;
  const void* x[2];  // keys, values (write: inputs; either may be null)
  void* y[2];        // read: outputs
  int64_t row[2], head[2];
  const int32_t* slots;
  int32_t* bad;
  int n, h_kv, page_shift, n_slots;
  int kind0;  // kind of blockIdx.z = 0 (0 keys, 1 values)
};

// Byte offset of the tile that holds `slot` for head h.
template <int D>
__device__ __forceinline__ size_t tile_offset(int slot, int h, int h_kv, int page_shift) {
  const int page = slot >> page_shift, in_page = slot & ((1 << page_shift) - 1);
  return (((size_t)page * h_kv + h << (page_shift - 4)) + (in_page >> 4)) * KvpTile<D>::kBytes;
}

// NaN to 0, everything else into +-kKvpLimit.
__device__ __forceinline__ float tame(float x) {
  return isnan(x) ? 0.f : fminf(fmaxf(x, -kKvpLimit), kKvpLimit);
}

// The smaller of two values, a NaN if either is one.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float rcp(float x) {  // to 2^-23 of itself
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The step of a group whose values span lo .. hi, fp16((hi - lo) / 15) in one
// rounding from fp64.  In fp32 the quotient is within 2^-22 of itself of the
// fp64 one; where that could round to another fp16 it is taken in fp64.
__device__ __forceinline__ uint16_t step16(float lo, float hi) {
  const float x = (hi - lo) * (1.f / 15.f);
  const uint16_t a = __half_as_ushort(__float2half_rn(x * (1.f - 0x1p-21f)));
  const uint16_t b = __half_as_ushort(__float2half_rn(x * (1.f + 0x1p-21f)));
  return a == b ? a : group_grid((double)lo, (double)hi, 4).s16;
}

// The codes of 8 values as a word, floor((v - m) / s + 1/2) clamped to 0 .. 15
// as fp64 arithmetic decides.  fp32 finds 15 x, x = (v - m) / (15 s) saturated to
// [0, 1], to 5e-6 and rounds it to the nearest integer by adding 1.5 * 2^23, which
// leaves the code in the low mantissa bits.  Where some value is closer than 2e-5
// to a half (bf16 values are on a coarse grid: one word in 170) the side of the
// half is the sign of v - m - (k + 1/2) s, which a fused multiply-add gets right
// where v - m is exact; where it is not, fp64 decides.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint16_t s16, uint16_t m16) {
  if (s16 == 0) return 0u;
  constexpr float kMagic = 12582912.f;
  const float m = h2f(m16), s = h2f(s16), inv = rcp(15.f * s);
  uint32_t word = 0;
  bool near_half = false;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float x = __saturatef((v[i] - m) * inv);
    const float r = fmaf(x, 15.f, kMagic);
    near_half = near_half || fabsf(fmaf(x, 15.f, kMagic - r)) > 0.49998f;
    word += (__float_as_uint(r) - 0x4B400000u) << (4 * i);
  }
  if (!near_half) return word;
  word = 0;
  bool inexact = false;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float t = v[i] - m, back = t - v[i];
    inexact = inexact || (v[i] - (t - back)) - (m + back) != 0.f;
    const float x = __saturatef(t * inv), q = fmaf(x, 15.f, kMagic) - kMagic;
    const float half = fmaf(x, 15.f, -q) >= 0.f ? q + 0.5f : q - 0.5f;
    const float code = fmaf(-half, s, t) >= 0.f ? half + 0.5f : half - 0.5f;
    word |= (__float_as_uint(fminf(code, 15.f) + kMagic) & 15u) << (4 * i);
  }
  if (inexact) {
    Grid16 g;
    g.s16 = s16, g.m16 = m16, g.S = h2d(s16), g.M = h2d(m16);
    word = 0;
#pragma unroll 1
    for (int i = 0; i < 8; i++) {
      float x = v[0];
#pragma unroll
      for (int k = 1; k < 8; k++) x = i == k ? v[k] : x;
      word |= (uint32_t)nested_code((double)x, g, 0, 15) << (4 * i);
    }
  }
  return word;
}

template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldcg(p), b = __ldcg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at));
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

// blockIdx: (64 tokens, head, keys or values).  Bound by instructions, 22 per value
// (a third of them per group, in all four lanes): 8,192 tokens of 8 heads in 16 us
// (bf16, fp16; 44 MB) or 20 us (fp32; 78 MB).  Four CTAs per SM at 64 registers, with
// 20 to 24 bytes a thread spilled at d = 128: 10% faster than three at 68.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 4) kvp_write_kernel(const __grid_constant__ CacheArgs a) {
  using L = KvpTile<D>;
  constexpr int G = L::G;
  pdl_trigger();
  pdl_wait();
  const int kind = a.kind0 + blockIdx.z, h = blockIdx.y, c = threadIdx.x & 3;
  const int tok = blockIdx.x * kTokens + (threadIdx.x >> 2);
  const int slot = tok < a.n ? a.slots[tok] : -1;
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (!ok && slot != -1 && a.bad && c == 0 && h == 0 && blockIdx.z == 0) atomicAdd(a.bad, 1);
  float v[G][8];
#pragma unroll
  for (int g = 0; g < G; g++)
#pragma unroll
    for (int i = 0; i < 8; i++) v[g][i] = 0.f;
  if (ok) {
#pragma unroll
    for (int g = 0; g < G; g++) load8<T>(a.x[kind], tok * a.row[kind] + h * a.head[kind] + g * 32 + c * 8, v[g]);
  }
  uint8_t* tile = a.pool + (ok ? tile_offset<D>(slot, h, a.h_kv, a.page_shift) : 0);
  const int t = slot & 15;
  uint32_t grid = 0;  // (s, m) of group c, or of group c % 2 where there are two
#pragma unroll
  for (int g = 0; g < G; g++) {
    float lo = v[g][0], hi = v[g][0];
#pragma unroll
    for (int i = 1; i < 8; i++) lo = min_nan(lo, v[g][i]), hi = fmaxf(hi, v[g][i]);
    if (!(lo >= -kKvpLimit && hi <= kKvpLimit)) {  // a NaN makes lo one
      lo = INFINITY, hi = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        v[g][i] = tame(v[g][i]);
        lo = fminf(lo, v[g][i]), hi = fmaxf(hi, v[g][i]);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const uint16_t s16 = step16(lo, hi), m16 = __half_as_ushort(__float2half_rn(lo));
    const uint32_t word = codes8(v[g], s16, m16);
    if (ok)
      *reinterpret_cast<uint32_t*>(tile + (kind ? L::kValueCodes : L::kKeyCodes) + (g * 16 + t) * 16 + c * 4) = word;
    if (c == g) grid = (uint32_t)s16 | ((uint32_t)m16 << 16);
  }
  if (!ok || c >= G) return;
  if (kind) {
    uint16_t* vz = reinterpret_cast<uint16_t*>(tile + L::kValueGrid) + ((t >> 1) * G + c) * 4 + (t & 1);
    vz[0] = (uint16_t)(grid & 0xffff), vz[2] = (uint16_t)(grid >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(tile + L::kKeyGrid + (t * G + c) * 4) = grid;
  }
}

// Bound by HBM: 131,072 tokens of 8 heads to bf16 or fp16, 705 MB in 120 us = 5.9 TB/s;
// to fp32, 1,242 MB in 274 us = 4.5 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kvp_read_kernel(const __grid_constant__ CacheArgs a) {
  using L = KvpTile<D>;
  constexpr int G = L::G;
  pdl_trigger();
  pdl_wait();
  const int kind = a.kind0 + blockIdx.z, h = blockIdx.y, c = threadIdx.x & 3;
  const int tok = blockIdx.x * kTokens + (threadIdx.x >> 2);
  if (tok >= a.n) return;
  const int slot = a.slots[tok];
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (!ok && slot != -1 && a.bad && c == 0 && h == 0 && blockIdx.z == 0) atomicAdd(a.bad, 1);
  uint32_t word[G], s[G], m[G];  // fp16 bits
#pragma unroll
  for (int g = 0; g < G; g++) word[g] = s[g] = m[g] = 0u;
  if (ok) {
    const uint8_t* tile = a.pool + tile_offset<D>(slot, h, a.h_kv, a.page_shift);
    const int t = slot & 15;
#pragma unroll
    for (int g = 0; g < G; g++)
      word[g] = *reinterpret_cast<const uint32_t*>(tile + (kind ? L::kValueCodes : L::kKeyCodes) + (g * 16 + t) * 16 +
                                                   c * 4);
    if (kind) {
      const uint4* p = reinterpret_cast<const uint4*>(tile + L::kValueGrid + (t >> 1) * (8 * G));
      const int sh = (t & 1) * 16;
#pragma unroll
      for (int g = 0; g < G; g += 2) {
        const uint4 z = p[g / 2];
        s[g] = z.x >> sh, m[g] = z.y >> sh, s[g + 1] = z.z >> sh, m[g + 1] = z.w >> sh;
      }
    } else {
      const uint2* p = reinterpret_cast<const uint2*>(tile + L::kKeyGrid + t * (4 * G));
#pragma unroll
      for (int g = 0; g < G; g += 2) {
        const uint2 z = p[g / 2];
        s[g] = z.x, m[g] = z.x >> 16, s[g + 1] = z.y, m[g + 1] = z.y >> 16;
      }
    }
  }
  const int64_t at = ((int64_t)tok * a.h_kv + h) * D + c * 8;
#pragma unroll
  for (int g = 0; g < G; g++) {
    const float sf = h2f((uint16_t)s[g]), mf = h2f((uint16_t)m[g]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = fmaf((float)((word[g] >> (4 * i)) & 15u), sf, mf);
    store8<T>(a.y[kind], at + g * 32, v);
  }
}

template <typename T>
sf_status launch_cache(const CacheArgs& a, int d, int kinds, bool read, cudaStream_t s) {
  const dim3 grid((a.n + kTokens - 1) / kTokens, a.h_kv, kinds);
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
