// kvp_decode.cu -- attention over the paged 4-bit cache for sequences with few
// query rows (rows = query tokens x query heads of one KV head): single-token
// decode, a handful of drafted tokens.
//
// One pass over the visible tokens with a running softmax.  The cache's bytes
// bound it (160 per token and KV head at d = 128), so the rest is built to stay
// under them: about 300 warp instructions per 16 tokens.  In its main loop a
// scheduler takes 500 cycles per tile of 16 tokens, where HBM gives one every 450.
// 8 sequences of 32,769 tokens, 8 KV and 32 query heads: 336 MB in 73 us =
// 4.6 TB/s; one of 131,072: 168 MB in 42 us = 4.0 TB/s; one of 8,192: 11 us, of
// which 2.3 go to finding the ranges, 3 to the merge kernel, 1.5 to the first
// loads.
//   - Tensor cores (m16n8k16) with the tokens as rows and the query rows as the
//     8 columns: S^T = K Q^T, O^T = V^T P^T.  tcgen05 tiles would be 128 rows
//     of which a decode step fills 4 to 8.
//   - Codes: a key's 4-bit code masked out of its word in place is the fp16
//     subnormal code * 2^-24 (low nibble of a byte) or code * 2^-20 (high
//     nibble), exact operands with no conversion; the queries of the high
//     nibbles carry the 1/16.  The group's step multiplies the fp32 sums, and
//     sum_g m_g (sum of q over g) is one more product whose A operand is the
//     stored grid itself.  So logits see no rounding but fp32 sums (queries
//     are scaled by a power of two to use fp16's range; the sums over a group
//     are split in two fp16).
//   - Values: (1024 + code) - 1024 and s code + m in fp16 pairs; one rounding of
//     the value to fp16, as a 16-bit cache would have.  The weights are rounded
//     to fp16 scaled so that the largest is near 2^15.  (fp16 outputs are then
//     2.5e-4 to 3.2e-4 from fp64, of which their own rounding is 2.1e-4; to keep
//     the low halves too would take three products for each of these.)
//   - ldmatrix reads the tiles as they lie (kvp.cuh); movmatrix turns the
//     weights from S^T's layout to the operand's.
//   - The running maximum moves only when some logit passes it by 2^6: then the
//     sums are rescaled, otherwise a step costs one vote.
// The work is cut into equal ranges on the device (kvp_attend.cuh).
#include <algorithm>

#include "kvp_attend.cuh"

namespace sf {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStepTiles = 2;  // tiles per warp and step
// An item's queries, join and output take about as long as 8 steps of the CTA
// (with 2, 8 and 12, bf16: 64 windows of 1,024 tokens 34.2, 33.9, 33.8 us; 100
// sequences of 200 to 3,000 tokens 64.0, 57.4, 57.5; 200 of 60 to 500, d = 64: 32.5,
// 27.5, 27.5; 8 of 32,769: 74.0, 72.9, 73.0).
constexpr int kExtra = 8;
constexpr float kRefGap = 6.f;   // log2: how far a logit may pass the reference
constexpr float kRefShift = 9.f; // weights are 2^(x - reference + 9) <= 2^15

// CTAs per SM: three while a thread's sums fit in 168 registers, two beyond (two
// columns: 27 us against 31 with three CTAs and their spilled registers).  At d = 128
// four columns still spill 324 bytes a thread (at d = 64 72 bytes), three 12.
constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }
constexpr int stages(int nt) { return nt == 4 ? 4 : 3; }  // four rows' columns need the fourth for the exchange

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStages = stages(NT);
  static constexpr int kStageBytes = kStepTiles * KvpTile<D>::kBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kOutStride = D + 8;  // floats per row in the warps' exchange
  static constexpr int kQBytes = NT > 1 ? NT * (D / 32) * 2 * 32 * 8 : 0;
  static constexpr int kSmem = kWarps * kWarpBytes + kQBytes;
  static_assert(kRows * kOutStride * 4 <= kWarpBytes, "the exchange reuses the stages");
  // a part of an item: sums [rows][D], then (reference, weight sum) per row
  static constexpr int kPartFloats = kRows * D + 2 * kRows;
};

struct DecodeArgs {
  KvpAttendArgs a;
  float* parts;     // [2 * ctas][part floats]
  // an item's entry: at (item number), written by the CTA with its first step,
  // where every item has one (no cu_q) and they are fewer than the CTAs; else at
  // that CTA, each CTA clearing its own before it starts
  KvpShared* desc;
  int by_item;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes, of which the last 16 - bytes are zeros.
__device__ __forceinline__ void cp_async16(uint32_t smem, const void* gmem, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a sum: nothing to add to.
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// ---- the kernel -------------------------------------------------------------

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT)) kvp_decode_kernel(const __grid_constant__ DecodeArgs da) {
  using L = KvpTile<D>;
  using C = Cfg<D, NT>;
  constexpr int G = L::G, MT = D / 16;
  const KvpAttendArgs& a = da.a;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ KvpRangeShared<KvpItem<C::kRows, kStepTiles, kExtra, true>> range_sh;
  // first token of a staged tile, low bit: all rows see all of it; negative: nothing there
  __shared__ __align__(8) int place[kWarps][C::kStages][kStepTiles];
  __shared__ float2 ml[kWarps][C::kRows];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, c = lane & 3;

  KvpItem<C::kRows, kStepTiles, kExtra, true> it;
  const KvpRange range = kvp_range<kThreads, false>(a, kWarps, range_sh, it);  // at least a step per warp
  if (tid == 0 && !da.by_item) da.desc[blockIdx.x].parts = 0;
  if (range.u0 == range.u1) return;
  const long u0 = range.u0, u1 = range.u1;
  long at = range.at;

  uint8_t* stage0 = smem + warp * C::kWarpBytes;
  const uint32_t stage0_u = smem_u32(stage0);
  uint2* qs = reinterpret_cast<uint2*>(smem + kWarps * C::kWarpBytes);  // NT > 1: the query operands

  for (;; at = it.end(at), it.next(a)) {  // this CTA's part of each item
    const int2 my = it.part(at, u0, u1);
    const int s0 = my.x, s1 = my.y;
    if (s0 == s1) break;  // the range ends before the item's first step
    const int rows_left = it.seq.n * a.group - it.rt * C::kRows, rows = min(rows_left, C::kRows);
    const int base = it.seq.len - it.seq.n, row0 = it.rt * C::kRows;
    const int32_t* pages = a.pages + (long)it.b * a.max_pages;

    // ---- the warp's steps s0 + warp, + kWarps, ...: lane l looks 32 steps
    // ahead for the place in the pool (in tiles) and in the sequence of its step's tiles
    const int my_steps = s1 - s0 > warp ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;
    uint32_t at_pool[kStepTiles];
    int at_seq[kStepTiles];
    auto look = [&](int k0) {
      const int step = s0 + warp + (k0 + lane) * kWarps;
#pragma unroll
      for (int j = 0; j < kStepTiles; j++) {
        const int i = step * kStepTiles + j;
        at_pool[j] = 0, at_seq[j] = -16;
        if (k0 + lane < my_steps && i < it.span.tiles) {
          const int t = it.span.tile(i), page = pages[t >> (a.page_shift - 4)];
          if (page >= 0 && page < a.n_pages) {
            at_pool[j] = ((uint32_t)(page * a.h_kv + it.g) << (a.page_shift - 4)) + (t & ((1 << (a.page_shift - 4)) - 1));
            at_seq[j] = t * 16 | (kvp_sees_all(a, it.span.p0, it.span.p1, t * 16, 16) ? 1 : 0);
          } else {
            kvp_note_bad(a.bad);
          }
        }
      }
    };
    int put_st = 0;
    auto fetch = [&](int k) {  // copy the tiles of the warp's step k into the next stage
      if (k < my_steps) {
        if ((k & 31) == 0) look(k);
        const uint32_t dst = stage0_u + put_st * C::kStageBytes + lane * 16;
        const uint8_t* src[kStepTiles];
        int where[kStepTiles], bytes[kStepTiles];
#pragma unroll
        for (int j = 0; j < kStepTiles; j++) {
          src[j] = a.pool + (size_t)__shfl_sync(0xffffffffu, at_pool[j], k & 31) * L::kBytes + lane * 16;
          where[j] = __shfl_sync(0xffffffffu, at_seq[j], k & 31);
          bytes[j] = where[j] >= 0 ? 16 : 0;  // nothing there: zeros
        }
        if (lane == 0) *reinterpret_cast<int2*>(&place[warp][put_st][0]) = make_int2(where[0], where[1]);
        constexpr int kChunks = L::kBytes / 16;  // 16-byte pieces per tile: 160 or 80
#pragma unroll
        for (int i = 0; i < kStepTiles * kChunks / 32; i++) {
          const bool second = lane + 32 * i >= kChunks;
          cp_async16(dst + 32 * i * 16, second ? src[1] + (32 * i - kChunks) * 16 : src[0] + 32 * i * 16,
                     second ? bytes[1] : bytes[0]);
        }
        if (++put_st == C::kStages) put_st = 0;
      }
      cp_commit();
    };
#pragma unroll
    for (int k = 0; k < C::kStages - 1; k++) fetch(k);

    // ---- query operands.  Row 8 nt + gid: this lane's elements 32 grp + 8 c + (0..7)
    uint32_t qf[NT > 1 ? 1 : G][2][2];  // [group][k-step][b0, b1]
    uint32_t qm[NT][2];                 // sums over group c, high and low part
    float k1[NT][2], k2[NT][2];         // factors of the rows 8 nt + 2 c, + 1
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const int r = 8 * nt + gid;
      float v[G][8];
      float top = 0.f;
      if (r < rows) {
        const int i = kvp_by_group(a, row0 + r), h = it.g * a.group + row0 + r - kvp_by_group(a, row0 + r) * a.group;
        const T* qr = static_cast<const T*>(a.q) + (it.seq.q0 + i) * a.q_row + h * a.q_head + 8 * c;
#pragma unroll
        for (int grp = 0; grp < G; grp++) {
          const uint4 w = *reinterpret_cast<const uint4*>(qr + 32 * grp);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float2 f = Elem<T>::to_float2(ws[e]);
            v[grp][2 * e] = f.x, v[grp][2 * e + 1] = f.y;
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      } else {
#pragma unroll
        for (int grp = 0; grp < G; grp++)
#pragma unroll
          for (int e = 0; e < 8; e++) v[grp][e] = 0.f;
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // power of two that takes the largest element to [2^10, 2^11)
      const int e = min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -100), 100);
      const float up = __uint_as_float((uint32_t)(127 + 10 - e) << 23);
      float sums[G];
#pragma unroll
      for (int grp = 0; grp < G; grp++) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; k++) v[grp][k] *= up, sum += v[grp][k];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sums[grp] = sum * 0.25f;  // |sum| < 2^14
        uint32_t f[2][2];
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
          f[ks][0] = pack2(v[grp][2 * ks], v[grp][2 * ks + 4]);
          f[ks][1] = pack2(v[grp][2 * ks + 1] * 0.0625f, v[grp][2 * ks + 5] * 0.0625f);
        }
        if constexpr (NT > 1) {
          if (warp == 0) {
            qs[((nt * G + grp) * 2 + 0) * 32 + lane] = make_uint2(f[0][0], f[0][1]);
            qs[((nt * G + grp) * 2 + 1) * 32 + lane] = make_uint2(f[1][0], f[1][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < 2; ks++) qf[grp][ks][0] = f[ks][0], qf[grp][ks][1] = f[ks][1];
        }
      }
      float sc = 0.f;
#pragma unroll
      for (int grp = 0; grp < G; grp++)
        if (c == grp) sc = sums[grp];
      const __half hi = __float2half_rn(sc), lo = __float2half_rn(sc - __half2float(hi));
      qm[nt][0] = (uint32_t)__half_as_ushort(hi) << 16, qm[nt][1] = (uint32_t)__half_as_ushort(lo) << 16;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int er = __shfl_sync(0xffffffffu, e, 4 * (2 * c + k));
        const float back = __uint_as_float((uint32_t)(127 - 10 + er) << 23) * a.scale_log2;
        k1[nt][k] = back * 16777216.f, k2[nt][k] = back * 4.f;
        const int rr = min(8 * nt + 2 * c + k, rows - 1);
        pos[nt][k] = base + kvp_by_group(a, row0 + rr);
      }
    }
    if constexpr (NT > 1) __syncthreads();

    float o[NT][MT][4], lsum[NT][2], ref[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int k = 0; k < 4; k++) o[nt][mt][k] = 0.f;
      lsum[nt][0] = lsum[nt][1] = 0.f;
      ref[nt][0] = ref[nt][1] = -INFINITY;
    }

    int st = 0;
    for (int k = 0; k < my_steps; k++) {
      cp_wait<C::kStages - 2>();
      __syncwarp();  // the step's tiles are there, and the stage of the step before is free
      fetch(k + C::kStages - 1);
      const uint32_t sb = stage0_u + st * C::kStageBytes;
      const uint8_t* sp = stage0 + st * C::kStageBytes;

      // ---- logits (log2 units): tokens gid, gid + 8 of each tile, rows 8 nt + 2 c, + 1
      float x[kStepTiles][NT][4];
      const int2 pl = *reinterpret_cast<const int2*>(&place[warp][st][0]);
      const int tb[kStepTiles] = {pl.x & ~1, pl.y & ~1};
      const bool whole = pl.x & pl.y & 1;
#pragma unroll
      for (int j = 0; j < kStepTiles; j++) {
        const uint32_t tile = sb + j * L::kBytes;
        const uint8_t* tp = sp + j * L::kBytes;
        // the token's steps, and its grid as an operand
        float s[2][G];
        uint32_t za[2];
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
          const uint8_t* zp = tp + L::kKeyGrid + (gid + 8 * hf) * (4 * G);
          uint32_t z[G];
          if constexpr (G == 4) {
            const uint4 z4 = *reinterpret_cast<const uint4*>(zp);
            z[0] = z4.x, z[1] = z4.y, z[2] = z4.z, z[3] = z4.w;
          } else {
            const uint2 z2 = *reinterpret_cast<const uint2*>(zp);
            z[0] = z2.x, z[1] = z2.y;
          }
#pragma unroll
          for (int grp = 0; grp < G; grp++) s[hf][grp] = __low2float(as_h2(z[grp]));
          za[hf] = c < G ? *reinterpret_cast<const uint32_t*>(zp + 4 * c) : 0u;
        }
        float xm[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) mma0(xm[nt], za[0], za[1], za[0], za[1], qm[nt][0], qm[nt][1]);
#pragma unroll
        for (int g2 = 0; g2 < G; g2 += 2) {
          uint32_t w[4];  // [group g2: tokens 0..7, 8..15; group g2 + 1: ...]
          ldsm4(w, tile + L::kKeyCodes + ((g2 + (lane >> 4)) * 16 + (lane & 15)) * 16);
#pragma unroll
          for (int gg = 0; gg < 2; gg++) {
            const int grp = g2 + gg;
            const uint32_t w0 = w[2 * gg], w1 = w[2 * gg + 1];
            const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
            uint32_t fa[2][4] = {{w0 & 0x000F000Fu, w1 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x00F000F0u},
                                 {v0 & 0x000F000Fu, v1 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x00F000F0u}};
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              float acc[4];
#pragma unroll
              for (int ks = 0; ks < 2; ks++) {
                uint32_t q0, q1;
                if constexpr (NT > 1) {
                  const uint2 qq = qs[((nt * G + grp) * 2 + ks) * 32 + lane];
                  q0 = qq.x, q1 = qq.y;
                } else {
                  q0 = qf[grp][ks][0], q1 = qf[grp][ks][1];
                }
                if (ks == 0)
                  mma0(acc, fa[ks][0], fa[ks][1], fa[ks][2], fa[ks][3], q0, q1);
                else
                  mma(acc, fa[ks][0], fa[ks][1], fa[ks][2], fa[ks][3], q0, q1);
              }
#pragma unroll
              for (int e = 0; e < 4; e++)
                x[j][nt][e] = grp == 0 ? s[e >> 1][grp] * acc[e] : fmaf(s[e >> 1][grp], acc[e], x[j][nt][e]);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int e = 0; e < 4; e++) x[j][nt][e] = fmaf(x[j][nt][e], k1[nt][e & 1], xm[nt][e] * k2[nt][e & 1]);
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < kStepTiles; j++)
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (tb[j] < 0 || !kvp_sees(a, pos[nt][e & 1], tb[j] + gid + 8 * (e >> 1))) x[j][nt][e] = -INFINITY;
      }

      // ---- running softmax: the reference moves only when a logit passes it by kRefGap
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
          float top = x[0][nt][kk];
#pragma unroll
          for (int j = 0; j < kStepTiles; j++) top = fmaxf(top, fmaxf(x[j][nt][kk], x[j][nt][kk + 2]));
          over = over || top > ref[nt][kk] + kRefGap;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int kk = 0; kk < 2; kk++) {
            float top = ref[nt][kk];
#pragma unroll
            for (int j = 0; j < kStepTiles; j++) top = fmaxf(top, fmaxf(x[j][nt][kk], x[j][nt][kk + 2]));
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
            const float f = top == -INFINITY ? 1.f : ex2(ref[nt][kk] - top);
            ref[nt][kk] = top;
            lsum[nt][kk] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; mt++) o[nt][mt][kk] *= f, o[nt][mt][kk + 2] *= f;
          }
      }
      uint32_t pb[kStepTiles][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        // a row that has seen nothing yet: weights 2^-inf = 0 against reference 0
        const float r0 = (ref[nt][0] == -INFINITY ? 0.f : ref[nt][0]) - kRefShift;
        const float r1 = (ref[nt][1] == -INFINITY ? 0.f : ref[nt][1]) - kRefShift;
#pragma unroll
        for (int j = 0; j < kStepTiles; j++) {
          const float p0 = ex2(x[j][nt][0] - r0), p1 = ex2(x[j][nt][1] - r1);
          const float p2 = ex2(x[j][nt][2] - r0), p3 = ex2(x[j][nt][3] - r1);
          lsum[nt][0] += p0 + p2, lsum[nt][1] += p1 + p3;
          pb[j][nt][0] = movm(pack2(p0, p1));
          pb[j][nt][1] = movm(pack2(p2, p3));
        }
      }

      // ---- values: rows dims 32 grp + 4 gid + (0..3), columns tokens 2 c, 2 c + 1, + 8
#pragma unroll
      for (int j = 0; j < kStepTiles; j++) {
        const uint32_t tile = sb + j * L::kBytes;
        const uint8_t* vz = sp + j * L::kBytes + L::kValueGrid;
        uint32_t zs[2][G], zm[2][G];
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
          const uint4* zp = reinterpret_cast<const uint4*>(vz + (c + 4 * hf) * (8 * G));
#pragma unroll
          for (int g2 = 0; g2 < G; g2 += 2) {
            const uint4 z = zp[g2 / 2];
            zs[hf][g2] = z.x, zm[hf][g2] = z.y, zs[hf][g2 + 1] = z.z, zm[hf][g2 + 1] = z.w;
          }
          if (!whole) {  // tokens that no row sees may hold anything: their grids count as 0
            const int t = tb[j] + 2 * c + 8 * hf;
            const uint32_t keep = (tb[j] >= 0 && kvp_some_sees(a, it.span.p0, it.span.p1, t) ? 0xffffu : 0u) |
                                  (tb[j] >= 0 && kvp_some_sees(a, it.span.p0, it.span.p1, t + 1) ? 0xffff0000u : 0u);
#pragma unroll
            for (int grp = 0; grp < G; grp++) zs[hf][grp] &= keep, zm[hf][grp] &= keep;
          }
        }
        const __half2 one16 = __float2half2_rn(0.0625f), off1 = __float2half2_rn(-1024.f),
                      off16 = __float2half2_rn(-64.f);
#pragma unroll
        for (int g2 = 0; g2 < G; g2 += 2) {
          uint32_t w[4];
          ldsm4t(w, tile + L::kValueCodes + ((g2 + (lane >> 4)) * 16 + (lane & 15)) * 16);
#pragma unroll
          for (int gg = 0; gg < 2; gg++) {
            const int grp = g2 + gg;
            uint32_t fa[2][4];  // [dims (0, 1) | (2, 3)][dim, token half]
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
              const __half2 s = as_h2(zs[hf][grp]), m = as_h2(zm[hf][grp]);
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const uint32_t ww = w[2 * gg + hf] >> (8 * e);
                const __half2 lo = __hadd2(as_h2((ww & 0x000F000Fu) | 0x64006400u), off1);
                const __half2 hi = __hfma2(as_h2((ww & 0x00F000F0u) | 0x64006400u), one16, off16);
                fa[e][2 * hf] = as_u32(__hfma2(lo, s, m));
                fa[e][2 * hf + 1] = as_u32(__hfma2(hi, s, m));
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
              for (int e = 0; e < 2; e++)
                mma(o[nt][2 * grp + e], fa[e][0], fa[e][1], fa[e][2], fa[e][3], pb[j][nt][0], pb[j][nt][1]);
          }
        }
      }
      if (++st == C::kStages) st = 0;
    }

    // ---- join the warps
    cp_wait<0>();
    __syncwarp();
    float* ex = reinterpret_cast<float*>(stage0);
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int kk = 0; kk < 2; kk++) {
        const int r = 8 * nt + 2 * c + kk;
        float l = lsum[nt][kk];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
        if (gid == 0) ml[warp][r] = make_float2(ref[nt][kk], l);
#pragma unroll
        for (int grp = 0; grp < G; grp++)
          *reinterpret_cast<float4*>(ex + r * C::kOutStride + 32 * grp + 4 * gid) =
              make_float4(o[nt][2 * grp][kk], o[nt][2 * grp][kk + 2], o[nt][2 * grp + 1][kk], o[nt][2 * grp + 1][kk + 2]);
      }
    __syncthreads();
    const bool all = s0 == 0 && s1 == it.steps;
    float* part = da.parts + (size_t)(2 * blockIdx.x + (s0 > 0 ? 0 : 1)) * C::kPartFloats;
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d4 = i % (D / 4) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; w++) top = fmaxf(top, ml[w][r].x);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const float2 m = ml[w][r];
        const float f = m.x == -INFINITY ? 0.f : ex2(m.x - top);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * C::kWarpBytes) +
                                                          r * C::kOutStride + d4);
        sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
        sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
        l = fmaf(f, m.y, l);
      }
      if (all) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: zeros
        const int qi = kvp_by_group(a, row0 + r), h = it.g * a.group + row0 + r - kvp_by_group(a, row0 + r) * a.group;
        T* out = static_cast<T*>(a.out) + ((size_t)(it.seq.q0 + qi) * a.h_q + h) * D + d4;
        *reinterpret_cast<uint2*>(out) =
            make_uint2(Elem<T>::from_float2(sum.x * inv, sum.y * inv), Elem<T>::from_float2(sum.z * inv, sum.w * inv));
      } else {
        *reinterpret_cast<float4*>(part + r * D + d4) = sum;
        if (d4 == 0) *reinterpret_cast<float2*>(part + C::kRows * D + 2 * r) = make_float2(top, l);
      }
    }
    // the CTA with the item's first step tells the merge kernel how many share it
    if (s0 == 0 && tid == 0 && (!all || da.by_item)) {
      KvpShared d;
      d.q_row = it.seq.q0, d.row0 = row0, d.rows = rows, d.head0 = it.g * a.group;
      d.parts = all ? 0 : kvp_sharers(range, it.end(at));
      d.cta = blockIdx.x;
      d.pad[0] = d.pad[1] = 0;
      da.desc[da.by_item ? (it.b * it.row_tiles(a, it.seq) + it.rt) * a.h_kv + it.g : blockIdx.x] = d;
    }
    __syncthreads();  // the exchange is read
    if (it.end(at) >= u1) break;
  }
}

// Joins the parts of an item: those of the CTA that has its first step (its
// second place) and of the CTAs after it (their first).  Part i goes to share i
// mod 2048 / D, the shares are summed and then added in order, whatever the form:
// a CTA takes ROWS rows of an item, 512 / ROWS threads a row, 4 elements and
// ROWS shares a thread.  With few items each row has a CTA of its own, so that
// its parts' loads are all under way at once.  A CTA whose rows all lie behind the
// item's leaves at once: so the row of a one-row CTA is known to exist (one query
// at 8192 tokens, the whole call: 11.4 -> 10.5 us).
constexpr int kMergeThreads = 512;

template <typename T, int D, int NT, int ROWS>
__global__ void __launch_bounds__(kMergeThreads) kvp_merge_kernel(const __grid_constant__ DecodeArgs da) {
  using C = Cfg<D, NT>;
  constexpr int kPer = kMergeThreads / ROWS, kShares = kMergeThreads / (D / 4), kThreadsPerElem = kPer / (D / 4);
  const KvpAttendArgs& a = da.a;
  __shared__ float4 sums[ROWS][kShares][D / 4];
  __shared__ float2 ls[ROWS][kShares];  // reference, weight sum
  pdl_trigger();
  pdl_wait();
  const KvpShared d = da.desc[blockIdx.x];
  const int rt = threadIdx.x / kPer, r = blockIdx.y * ROWS + rt, tid = threadIdx.x % kPer;
  if (d.parts == 0 || blockIdx.y * ROWS >= d.rows) return;
  const bool live = r < d.rows;
  const int q4 = tid % (D / 4);
#pragma unroll 1
  for (int share = tid / (D / 4); share < min(kShares, d.parts); share += kThreadsPerElem) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f, top = -INFINITY;
    if (live) {
      constexpr int kAhead = 4;
      for (int i0 = share; i0 < d.parts; i0 += kAhead * kShares) {
        float2 m[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
          const int i = i0 + k * kShares;
          m[k] = make_float2(-INFINITY, 0.f), v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < d.parts) {
            const float* p = da.parts + (size_t)(2 * (d.cta + i) + (i == 0 ? 1 : 0)) * C::kPartFloats;
            m[k] = *reinterpret_cast<const float2*>(p + C::kRows * D + 2 * r);
            v[k] = *reinterpret_cast<const float4*>(p + r * D + 4 * q4);
          }
        }
        float now = top;
#pragma unroll
        for (int k = 0; k < kAhead; k++) now = fmaxf(now, m[k].x);
        const float old = top == -INFINITY ? 0.f : ex2(top - now);
        sum.x *= old, sum.y *= old, sum.z *= old, sum.w *= old, l *= old;
        top = now;
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
          const float f = m[k].x == -INFINITY ? 0.f : ex2(m[k].x - top);
          sum.x = fmaf(f, v[k].x, sum.x), sum.y = fmaf(f, v[k].y, sum.y);
          sum.z = fmaf(f, v[k].z, sum.z), sum.w = fmaf(f, v[k].w, sum.w);
          l = fmaf(f, m[k].y, l);
        }
      }
    }
    sums[rt][share][q4] = sum;
    if (q4 == 0) ls[rt][share] = make_float2(top, l);
  }
  __syncthreads();
  if (tid >= D / 4 || !live) return;
  const int shares = min(kShares, d.parts);
  float top = -INFINITY, l = 0.f;
  for (int k = 0; k < shares; k++) top = fmaxf(top, ls[rt][k].x);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < shares; k++) {
    const float2 m = ls[rt][k];
    const float f = m.x == -INFINITY ? 0.f : ex2(m.x - top);
    const float4 v = sums[rt][k][q4];
    sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
    sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
    l = fmaf(f, m.y, l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int qi = kvp_by_group(a, d.row0 + r), h = d.head0 + d.row0 + r - qi * a.group;
  T* out = static_cast<T*>(a.out) + ((size_t)(d.q_row + qi) * a.h_q + h) * D + 4 * q4;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(Elem<T>::from_float2(sum.x * inv, sum.y * inv), Elem<T>::from_float2(sum.z * inv, sum.w * inv));
}

// Columns of 8 rows per item: as few as the rows need, in items of at most four.
// A column costs its products and softmax, every item the decoding of the cache
// (8 sequences of 8192 tokens, 4 KV heads, d = 128: 27 us with two columns, 32
// with three, 40 with four).
int row_blocks(int rows) {
  const int blocks = (rows + 7) / 8, items = (blocks + 3) / 4;
  return (blocks + items - 1) / items;
}
int decode_ctas(int nt) { return num_sms() * ctas_per_sm(nt); }

template <typename T, int D, int NT>
sf_status launch_decode(const KvpAttendArgs& a, cudaStream_t s) {
  using C = Cfg<D, NT>;
  const int ctas = decode_ctas(NT);
  DecodeArgs da;
  da.a = a;
  da.desc = static_cast<KvpShared*>(a.ws);
  da.parts = reinterpret_cast<float*>(da.desc + ctas);
  // without cu_q the rows of every sequence, and so the items, are known
  const long each = (long)(a.n_q / a.batch) * a.group;
  const int most = a.cu_q ? C::kRows : (int)std::min<long>(each, C::kRows);
  const long items = (each + C::kRows - 1) / C::kRows * a.h_kv * a.batch;
  da.by_item = !a.cu_q && items < ctas;
  const int entries = da.by_item ? (int)items : ctas;
  SF_CUDA((kvp_allow_smem<kvp_decode_kernel<T, D, NT>>(C::kSmem)));
  SF_CUDA(launch_pdl(kvp_decode_kernel<T, D, NT>, dim3(ctas), dim3(kThreads), C::kSmem, s, da));
  if ((long)entries * most <= 2l * num_sms())
    SF_CUDA(launch_pdl(kvp_merge_kernel<T, D, NT, 1>, dim3(entries, most), dim3(kMergeThreads), 0, s, da));
  else
    SF_CUDA(launch_pdl(kvp_merge_kernel<T, D, NT, 4>, dim3(entries, (most + 3) / 4), dim3(kMergeThreads), 0, s, da));
  return SF_OK;
}

template <typename T, int D>
sf_status launch_decode_nt(const KvpAttendArgs& a, int rows, cudaStream_t s) {
  switch (row_blocks(rows)) {
    case 1: return launch_decode<T, D, 1>(a, s);
    case 2: return launch_decode<T, D, 2>(a, s);
    case 3: return launch_decode<T, D, 3>(a, s);
    default: return launch_decode<T, D, 4>(a, s);
  }
}

}  // namespace

size_t kvp_decode_workspace(int d, int rows) {
  const int nt = row_blocks(rows), ctas = decode_ctas(nt);
  return (size_t)ctas * (sizeof(KvpShared) + 2 * (8 * nt * d + 16 * nt) * sizeof(float));
}

sf_status launch_kvp_decode(const KvpAttendArgs& a, int d, sf_dtype dtype, int rows, cudaStream_t s) {
  if (d == 128)
    return dtype == SF_F16 ? launch_decode_nt<__half, 128>(a, rows, s) : launch_decode_nt<__nv_bfloat16, 128>(a, rows, s);
  return dtype == SF_F16 ? launch_decode_nt<__half, 64>(a, rows, s) : launch_decode_nt<__nv_bfloat16, 64>(a, rows, s);
}

}  // namespace sf
