// kvp.cuh -- layout of the paged 4-bit KV cache (include/sf.h, sf_kvp) and the
// 16- and 32-bit element types its entry points take.
//
// A 16-token tile keeps, per group of 32 elements, 16 rows of 16 bytes: eight
// of them are one 8 x 8 matrix of 16-bit units for ldmatrix, 128 contiguous
// bytes and so free of bank conflicts.  Read as stored, a lane gets the eight
// nibbles of its quarter of a token's group (the query.key contraction runs
// over elements); read transposed, the same nibbles of two neighbouring tokens
// in the two halves of a register (the weight.value contraction runs over
// tokens).  Keys and values can therefore share one layout.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace sf {

constexpr int kKvpGroup = 32;   // elements that share a grid
constexpr int kKvpTile = 16;    // tokens per tile
constexpr float kKvpLimit = 65408.f;

template <int D>
struct KvpTile {
  static constexpr int G = D / kKvpGroup;
  static constexpr int kKeyCodes = 0;
  static constexpr int kValueCodes = 8 * D;
  static constexpr int kKeyGrid = 16 * D;
  static constexpr int kValueGrid = 18 * D;
  static constexpr int kBytes = 20 * D;
};

template <typename T>
struct Elem;
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float2 to_float2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  // a grid value can exceed the largest fp16 by its rounding only if the
  // inputs did: the clamp of sf_kvp keeps every stored value inside
  static __device__ __forceinline__ uint32_t from_float2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float2 to_float2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t from_float2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
};

// Host-side validation of the descriptor (kvp_cache.cu).
sf_status check_kvp(const sf_kvp* kv);

}  // namespace sf
