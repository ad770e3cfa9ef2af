// kvp_prefill.cu -- attention over the paged 4-bit cache for sequences with
// many query rows (prefill, prefill chunks behind a cached prefix).
//
// 4 d products per (row, token) against 1.25 d bytes per token make this a
// matrix problem: tcgen05 products of 128-row tiles with fp32 accumulators in
// TMEM.  Rows are query tokens x the query heads of one KV head, so that heads
// that share keys and values share their decoding.  A CTA takes 256 rows as two
// tiles and walks the visible cache 128 tokens at a time:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row.  S comes out of
//                   TMEM, the weights go back into S's columns as the fp16
//                   operand of the second product.  While one tile's weights
//                   are made the tensor core works for the other.
//   warps 8-15      decode 128 tokens' codes to fp16 keys and values in shared
//                   memory (128-byte swizzle), once for both tiles
//   warp 16         one thread issues the products
// Numerics: keys and values are rounded once to fp16, as a 16-bit cache would
// hold them; queries are scaled per row by a power of two into fp16's range
// (exact for fp16 and bf16 but for elements 2^24 below the row's largest);
// weights are rounded to fp16, scaled so that the largest is near 2^15; sums are
// fp32.  (fp16 outputs are then up to 8e-4 from fp64 in relative L2, 2.1e-4 being
// their own rounding, with keys of which some channels are ten times the others;
// the low halves of keys, values and weights would take two to three times the
// products.)  The softmax reference moves only when a logit passes it by 2^6, so
// the output sums are hardly ever rescaled.
//
// Elements of 8 are kept in the order (0 4 1 5 2 6 3 7), the order in which a
// masked code word gives them up: queries and keys alike, and the output's
// columns are put back in order when they are stored.
//
// What bounds it: each tile's chain of softmax (2,750 cycles for 128 tokens: 128
// exponentials a thread at 8 cycles and warp on the special-function unit, shared
// by two warps, are 1,700 of them) and products (1,800 for 16 that take 1,034 back
// to back).  Two tiles in turn keep the tensor cores 45% busy; TMEM has no room for
// a third.  32 bf16 heads (8 KV heads, d = 128): the last 2,048 queries at length
// 16,384 in 0.505 ms = 1.02 PFLOP/s; a prompt of 8,192 in 0.63 ms = 0.88; one of
// 4,096 with a window of 1,024 in 0.13 ms = 0.47 (an item's queries, first step and
// output cost 9 us and are not hidden).
//
// The work is cut into equal ranges on the device (kvp_attend.cuh); every wait
// is bounded.
#include "internal.cuh"
#include "kvp_attend.cuh"
#include "kvp_wait.cuh"

namespace sf {
namespace {

constexpr int kRows = 256, kTileRows = 128;
constexpr int kStep = 8;                 // cache tiles per step: 128 tokens
constexpr int kTokens = kStep * kKvpTile;
constexpr int kSoftWarps = 8, kFillWarps = 8;
constexpr int kThreads = (kSoftWarps + kFillWarps + 4) * 32;  // the last warpgroup issues the products
// Registers per thread: the launch's 96 x 640 threads = 480 x 128, given out anew
// as (2 x 160 + 2 x 56 + 48) x 128.  ptxas spills 256 bytes a thread at d = 128, 136
// at d = 64.
constexpr int kSoftRegs = 160, kFillRegs = 56, kIssueRegs = 48;
constexpr int kRing = 4;                 // steps whose token places are kept
constexpr float kRefGap = 6.f, kRefShift = 9.f;
constexpr int kMinSteps = 1;             // the fewest steps worth a CTA
// An item's queries and output take about as long as 4 steps (bf16, with 2, 4 and 9:
// prompts of 2,000 and 4,001 tokens, window 1,024: 205, 180, 178 us; 24 prompts of 300:
// 114, 110, 112; 2,048 queries at 16,384: 500, 493, 498; 100 queries at five lengths
// up to 2,000, d = 64: 36, 36, 41).
constexpr int kExtra = 4;

__device__ unsigned int g_wait_timeouts;

using Item = KvpItem<kRows, kStep, kExtra, false>;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;              // 64-element halves of a 128-byte swizzled row
  static constexpr int kTileBytes = kHalves * 16384;  // 128 rows
  static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = 4 * kTileBytes;
  static constexpr int kSmem = 6 * kTileBytes + 1024;  // + alignment
  static constexpr int kPartFloats = kRows * D + 2 * kRows;
};

struct PrefillArgs {
  KvpAttendArgs a;
  float* parts;     // [2 * ctas][part floats]
  // an item's entry: at (item number), written by the CTA with its first step,
  // where every item has one (no cu_q) and they are fewer than the CTAs; else at
  // that CTA, each CTA clearing its own before it starts
  KvpShared* desc;
  int by_item;
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- PTX --------------------------------------------------------------------

__device__ __forceinline__ void mbar_wait(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
  sf::mbar_wait(bar, parity, gave_up, &g_wait_timeouts);
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// One product step (K = 16).  The descriptors' upper halves are constants, the
// lower ones differ by constants: the whole warp computes them, so that they
// stay in uniform registers, and one elected lane issues.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t a_hi, uint32_t b_hi,
                                          uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %6, 0;\n mov.b64 da, {%1, %3};\n mov.b64 db, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                          uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %5, 0;\n mov.b64 db, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(is));
  return is != 0;
}
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// The loads are complete; the registers are named so that nothing that uses
// them moves above the wait.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) : : "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values in a register pair: one instruction for both.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// Descriptor of a 128-byte swizzled operand, 8-row groups 1024 bytes apart:
// lower half (address, `far`) and upper half.  Contraction along the rows'
// bytes (queries, keys): `far` is not used.  Contraction along the rows
// (values): 64-element halves lie `far` bytes apart.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t far) {
  return ((addr >> 4) & 0x3FFF) | ((far >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t mma_desc(int n, bool b_by_rows) {  // fp16 x fp16 -> fp32, M = 128
  return (1u << 4) | (b_by_rows ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// 8 codes of a word to fp16 values in the order (0 4)(1 5)(2 6)(3 7): 1024 +
// code by masking into the mantissa, minus 1024, times s, plus m.
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 s, __half2 m) {
  const __half2 one16 = __float2half2_rn(0.0625f), off1 = __float2half2_rn(-1024.f), off16 = __float2half2_rn(-64.f);
  const uint32_t v = w >> 8;
  uint4 r;
  r.x = as_u32(__hfma2(__hadd2(as_h2((w & 0x000F000Fu) | 0x64006400u), off1), s, m));
  r.y = as_u32(__hfma2(__hfma2(as_h2((w & 0x00F000F0u) | 0x64006400u), one16, off16), s, m));
  r.z = as_u32(__hfma2(__hadd2(as_h2((v & 0x000F000Fu) | 0x64006400u), off1), s, m));
  r.w = as_u32(__hfma2(__hfma2(as_h2((v & 0x00F000F0u) | 0x64006400u), one16, off16), s, m));
  return r;
}

// A warp's place in its CTA's work: kept in shared memory, so that it takes no
// registers while a part of an item is under way.
struct Walk {
  Item it;
  long at;
  int s0, s1;  // steps of the item; s0 == s1: the range is over

  __device__ __forceinline__ void cut(const KvpRange& r) {
    const int2 my = it.part(at, r.u0, r.u1);
    s0 = my.x, s1 = my.y;
  }
};

struct Control {
  uint64_t q_full[2], s_full[2], p_full[2], o_done[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], last;
  KvpRangeShared<Item> range_sh;
  KvpRange range;
  Walk walk[kThreads / 32];
  // first token of each cache tile of the step, low bit: all rows see all of
  // it; -16: nothing there
  alignas(16) int place[kRing][kStep];  // read four at a time
  uint32_t tmem;
  volatile int gave_up;
};

// Bit i: the row at position p sees token base + i (16 tokens).
__device__ __forceinline__ uint32_t seen16(const KvpAttendArgs& a, int p, int base) {
  if (base < 0) return 0;
  const auto below = [](int n) { return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1u; };  // bits 0 .. n-1
  uint32_t m = below(p - base + 1);
  if (a.window) m &= ~below(p - a.window + 1 - base) | below(a.sinks - base);
  return m;
}

// The same for two cache tiles' places (Control::place).
__device__ __forceinline__ uint32_t seen32(const KvpAttendArgs& a, int p, int place0, int place1) {
  return seen16(a, p, place0 & ~1) | (seen16(a, p, place1 & ~1) << 16);
}
__device__ __forceinline__ void hide(uint32_t (&s)[32], uint32_t seen) {
#pragma unroll
  for (int i = 0; i < 32; i++) s[i] = seen >> i & 1 ? s[i] : 0xff800000u;  // -infinity
}
__device__ __forceinline__ float largest(const uint32_t (&s)[32]) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; k++) m[k] = __uint_as_float(s[k]);
#pragma unroll
  for (int i = 4; i < 32; i += 8)
#pragma unroll
    for (int k = 0; k < 4; k++) {
      m[k] = fmaxf(m[k], __uint_as_float(s[i + k]));
      if (i + 4 < 32) m[k] = fmaxf(m[k], __uint_as_float(s[i + 4 + k]));
    }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) kvp_prefill_kernel(const __grid_constant__ PrefillArgs pa) {
  using L = KvpTile<D>;
  using C = Cfg<D>;
  constexpr int G = L::G;
  const KvpAttendArgs& a = pa.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control ctl;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t smem_at = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  if (tid == 0) {
    for (int t = 0; t < 2; t++) {
      mbar_init(&ctl.q_full[t], kTileRows), mbar_init(&ctl.o_done[t], 1);
      mbar_init(&ctl.s_full[t], 1), mbar_init(&ctl.p_full[t], kTileRows);
      mbar_init(&ctl.k_full[t], kFillWarps * 32), mbar_init(&ctl.k_empty[t], 1);
      mbar_init(&ctl.v_full[t], kFillWarps * 32), mbar_init(&ctl.v_empty[t], 1);
    }
    mbar_init(&ctl.last, 1);
    ctl.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  Walk& walk = ctl.walk[warp];
  {
    Item it;
    const KvpRange range = kvp_range<kThreads, true>(a, kMinSteps, ctl.range_sh, it);
    if (tid == 0) {
      ctl.range = range;
      if (!pa.by_item) pa.desc[blockIdx.x].parts = 0;
    }
    if (range.u0 == range.u1) return;
    if (lane == 0) {
      walk.it = it, walk.at = range.at;
      walk.cut(range);
    }
  }
  // to the next item; false at the end of the range
  auto advance = [&]() {
    __syncwarp();
    const bool more = walk.it.end(walk.at) < ctl.range.u1;
    __syncwarp();
    if (more && lane == 0) {
      walk.at = walk.it.end(walk.at);
      walk.it.next(a);
      walk.cut(ctl.range);
    }
    __syncwarp();
    return more && walk.s0 < walk.s1;
  };
  if (warp == kSoftWarps + kFillWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = ctl.tmem;  // columns: S tile 0, S tile 1 (128 each), O tile 0, O tile 1 (D each)
  int step_no = 0;  // steps of this CTA so far, over all segments

  if (warp < kSoftWarps) {
    regs_up<kSoftRegs>();
    // ======================= softmax: a row per thread ========================
    const int t = warp >> 2, tr = tid & 127, r = t * kTileRows + tr;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp & 3)
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * D;
    int n_s = 0, n_o = 0;  // phases of s_full, o_done
    if (walk.s0 < walk.s1) do {
      const int s0 = walk.s0, s1 = walk.s1;
      const int row0 = walk.it.rt * kRows, rows = min(walk.it.seq.n * a.group - row0, kRows);
      if (t == 0 || rows > kTileRows) {
        const int rr = row0 + min(r, rows - 1);
        const int pos = walk.it.seq.len - walk.it.seq.n + kvp_by_group(a, rr);
        // ---- the tile's queries: D / 8 lanes a row, each row scaled by a power
        // of two into fp16's range.  A negative scale turns the query around and
        // a scale of 0 becomes one that rounds away, so that the largest S is
        // the largest logit.
        constexpr int kLanes = D / 8, kPerWarp = 32 / kLanes;  // lanes a row, rows at a time
        uint4 w[kLanes];
        const int part8 = lane % kLanes, first_row = t * kTileRows + (warp & 3) * 32 + lane / kLanes;
#pragma unroll
        for (int i = 0; i < kLanes; i++) {
          const int x = row0 + min(first_row + i * kPerWarp, rows - 1);
          w[i] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                      (walk.it.seq.q0 + kvp_by_group(a, x)) * a.q_row +
                                                      (walk.it.g * a.group + x - kvp_by_group(a, x) * a.group) * a.q_head) + part8);
        }
        int my_e = 0;
#pragma unroll
        for (int i = 0; i < kLanes; i++) {
          const float2 f0 = Elem<T>::to_float2(w[i].x), f1 = Elem<T>::to_float2(w[i].y);
          const float2 f2 = Elem<T>::to_float2(w[i].z), f3 = Elem<T>::to_float2(w[i].w);
          float top = fmaxf(fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))),
                            fmaxf(fmaxf(fabsf(f2.x), fabsf(f2.y)), fmaxf(fabsf(f3.x), fabsf(f3.y))));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = min(max((int)((__float_as_uint(top) >> 23) & 255) - 127, -100), 100);
          const int qrow = first_row + i * kPerWarp;
          const float up = qrow < rows ? copysignf(__uint_as_float((uint32_t)(127 + 10 - e) << 23), a.scale_log2) : 0.f;
          uint4 o;
          o.x = pack2(f0.x * up, f2.x * up), o.y = pack2(f0.y * up, f2.y * up);
          o.z = pack2(f1.x * up, f3.x * up), o.w = pack2(f1.y * up, f3.y * up);
          const int in_tile = qrow - t * kTileRows;
          *reinterpret_cast<uint4*>(smem + C::kQ + t * C::kTileBytes + (part8 >> 3) * 16384 + in_tile * 128 +
                                    (((part8 & 7) ^ (in_tile & 7)) << 4)) = o;
          // lane x of the warp owns row x: its exponent lies with the lanes of that row
          const int theirs = __shfl_sync(0xffffffffu, e, (lane % kPerWarp) * kLanes);
          if (lane / kPerWarp == i) my_e = theirs;
        }
        const float kappa = fmaxf(__uint_as_float((uint32_t)(127 - 10 + my_e) << 23) * fabsf(a.scale_log2), 1e-37f);
        fence_async_smem();
        tc_before();
        mbar_arrive(&ctl.q_full[t]);

        float ref = -INFINITY, l = 0.f;
        for (int j = s0; j < s1; j++) {
          mbar_wait(&ctl.s_full[t], n_s & 1, &ctl.gave_up);
          __syncwarp();
          n_s++;
          tc_after();
          const int ring = (step_no + j - s0) & (kRing - 1);
          const int4 pl0 = *reinterpret_cast<const int4*>(&ctl.place[ring][0]);
          const int4 pl1 = *reinterpret_cast<const int4*>(&ctl.place[ring][4]);
          const int place[kStep] = {pl0.x, pl0.y, pl0.z, pl0.w, pl1.x, pl1.y, pl1.z, pl1.w};
          const bool whole = (place[0] & place[1] & place[2] & place[3] & place[4] & place[5] & place[6] & place[7]) & 1;
          uint32_t s[kTokens / 32][32];
#pragma unroll
          for (int ch = 0; ch < kTokens / 32; ch++) tc_ld32(s[ch], s_at + ch * 32);
          tc_wait_ld(s[0]), tc_wait_ld(s[1]), tc_wait_ld(s[2]), tc_wait_ld(s[3]);
          if (!whole) {
#pragma unroll
            for (int ch = 0; ch < kTokens / 32; ch++)
              hide(s[ch], seen32(a, pos, place[2 * ch], place[2 * ch + 1]));
          }
          const float top = fmaxf(fmaxf(largest(s[0]), largest(s[1])), fmaxf(largest(s[2]), largest(s[3]))) * kappa;
          if (__any_sync(0xffffffffu, top > ref + kRefGap)) {
            const float next = fmaxf(ref, top);
            const float f = next == -INFINITY ? 1.f : ex2(ref - next);
            ref = next;
            l *= f;
            if (j > s0) {  // the products into O so far are complete: S was issued after them
#pragma unroll
              for (int ch = 0; ch < D / 16; ch++) {
                uint32_t o[16];
                tc_ld16(o, o_at + ch * 16);
                tc_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tc_st16(o_at + ch * 16, o);
              }
            }
          }
          const float off = kRefShift - (ref == -INFINITY ? 0.f : ref);
          uint64_t sum0 = 0, sum1 = 0;  // two fp32 sums each
          const uint64_t kk = pair(kappa, kappa), oo = pair(off, off);
#pragma unroll
          for (int ch = 0; ch < kTokens / 32; ch++) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float2 y0 = split(fma2(pair(__uint_as_float(s[ch][i]), __uint_as_float(s[ch][i + 1])), kk, oo));
              const float2 y1 = split(fma2(pair(__uint_as_float(s[ch][i + 2]), __uint_as_float(s[ch][i + 3])), kk, oo));
              const float p0 = ex2(y0.x), p1 = ex2(y0.y), p2 = ex2(y1.x), p3 = ex2(y1.y);
              sum0 = add2(sum0, pair(p0, p1)), sum1 = add2(sum1, pair(p2, p3));
              p[i / 2] = pack2(p0, p1), p[i / 2 + 1] = pack2(p2, p3);
            }
            tc_st16(s_at + ch * 16, p);
          }
          const float2 sum = split(add2(sum0, sum1));
          l += sum.x + sum.y;
          tc_wait_st();
          tc_before();
          mbar_arrive(&ctl.p_full[t]);
        }

        // ---- the row's output, or its part of it
        mbar_wait(&ctl.o_done[t], n_o++ & 1, &ctl.gave_up);
        __syncwarp();
        tc_after();
        const bool all = s0 == 0 && s1 == walk.it.steps;
        float* part = pa.parts + (size_t)(2 * blockIdx.x + (s0 > 0 ? 0 : 1)) * C::kPartFloats;
        const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: zeros
        T* out = static_cast<T*>(a.out) +
                 ((size_t)(walk.it.seq.q0 + kvp_by_group(a, rr)) * a.h_q + walk.it.g * a.group + rr - kvp_by_group(a, rr) * a.group) * D;
#pragma unroll
        for (int ch = 0; ch < D / 32; ch++) {
          uint32_t o[32];
          tc_ld32(o, o_at + ch * 32);
          tc_wait_ld(o);
          if (r < rows) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 4; i++) v[i] = __uint_as_float(o[k + 2 * i]), v[i + 4] = __uint_as_float(o[k + 2 * i + 1]);
              if (all) {
                uint4 w;
                w.x = Elem<T>::from_float2(v[0] * inv, v[1] * inv), w.y = Elem<T>::from_float2(v[2] * inv, v[3] * inv);
                w.z = Elem<T>::from_float2(v[4] * inv, v[5] * inv), w.w = Elem<T>::from_float2(v[6] * inv, v[7] * inv);
                *reinterpret_cast<uint4*>(out + ch * 32 + k) = w;
              } else {
                float4* w = reinterpret_cast<float4*>(part + r * D + ch * 32 + k);
                w[0] = make_float4(v[0], v[1], v[2], v[3]);
                w[1] = make_float4(v[4], v[5], v[6], v[7]);
              }
            }
          }
        }
        if (!all && r < rows) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(ref, l);
        if (s0 == 0 && tid == 0 && (!all || pa.by_item)) {
          KvpShared d;
          d.q_row = walk.it.seq.q0, d.row0 = row0, d.rows = rows, d.head0 = walk.it.g * a.group;
          d.parts = all ? 0 : kvp_sharers(ctl.range, walk.it.end(walk.at));
          d.cta = blockIdx.x;
          d.pad[0] = d.pad[1] = 0;
          pa.desc[pa.by_item ? (walk.it.b * Item::row_tiles(a, walk.it.seq) + walk.it.rt) * a.h_kv + walk.it.g
                             : blockIdx.x] = d;
        }
      }
      step_no += s1 - s0;
    } while (advance());
  } else if (warp < kSoftWarps + kFillWarps) {
    regs_down<kFillRegs>();
    // ======================= decoding: half a token's groups per thread =======
    constexpr int H = G / 2;
    const int tk = tid & 127, sub = tk >> 4, tt = tk & 15, g0 = (warp - kSoftWarps) / 4 * H;
    uint4 kc[H], vc[H], vz;  // codes; value grids (one or two groups)
    uint2 kz;                // key grids
    if (walk.s0 < walk.s1) do {
      const int s0 = walk.s0, s1 = walk.s1;
      const int32_t* pages = a.pages + (long)walk.it.b * a.max_pages;
      // the page entry of this thread's cache tile of a step (-1: none), and the tile's address
      auto entry = [&](int step) {
        const int i = step * kStep + sub;
        if (step >= s1 || i >= walk.it.span.tiles) return -1;
        const int page = pages[walk.it.span.tile(i) >> (a.page_shift - 4)];
        if (page >= 0 && page < a.n_pages) return page;
        if (tt == 0 && g0 == 0) kvp_note_bad(a.bad);
        return -1;
      };
      auto tile_of = [&](int page, int step) -> const uint8_t* {
        if (page < 0) return nullptr;
        const int in_page = walk.it.span.tile(step * kStep + sub) & ((1 << (a.page_shift - 4)) - 1);
        return a.pool + ((((size_t)page * a.h_kv + walk.it.g) << (a.page_shift - 4)) + in_page) * L::kBytes;
      };
      auto load_k = [&](const uint8_t* p) {
#pragma unroll
        for (int g = 0; g < H; g++) kc[g] = make_uint4(0, 0, 0, 0);
        kz = make_uint2(0, 0);
        if (!p) return;
#pragma unroll
        for (int g = 0; g < H; g++)
          kc[g] = __ldcg(reinterpret_cast<const uint4*>(p + L::kKeyCodes + ((g0 + g) * 16 + tt) * 16));
        const uint8_t* z = p + L::kKeyGrid + (tt * G + g0) * 4;
        if constexpr (H == 2)
          kz = __ldcg(reinterpret_cast<const uint2*>(z));
        else
          kz.x = __ldcg(reinterpret_cast<const unsigned int*>(z));
      };
      auto load_v = [&](const uint8_t* p) {
#pragma unroll
        for (int g = 0; g < H; g++) vc[g] = make_uint4(0, 0, 0, 0);
        vz = make_uint4(0, 0, 0, 0);
        if (!p) return;
#pragma unroll
        for (int g = 0; g < H; g++)
          vc[g] = __ldcg(reinterpret_cast<const uint4*>(p + L::kValueCodes + ((g0 + g) * 16 + tt) * 16));
        const uint8_t* z = p + L::kValueGrid + ((tt >> 1) * G + g0) * 8;
        if constexpr (H == 2) {
          vz = __ldcg(reinterpret_cast<const uint4*>(z));
        } else {
          const uint2 zz = __ldcg(reinterpret_cast<const uint2*>(z));
          vz.x = zz.x, vz.y = zz.y;
        }
      };
      // where this thread's first 16 bytes go in a tile; the others by xor
      const uint32_t row_at = (g0 >> 1) * 16384 + tk * 128, swz = (((g0 & 1) * 4) ^ (tk & 7)) << 4;
      auto put = [&](uint8_t* dst, int g, const uint4& codes, __half2 s, __half2 m) {
        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
        for (int i = 0; i < 4; i++)
          *reinterpret_cast<uint4*>(dst + row_at + (swz ^ ((g * 4 + i) << 4))) = decode8(w[i], s, m);
      };
      int page_next = entry(s0 + 1);
      const uint8_t* tile = tile_of(entry(s0), s0);
      load_k(tile);
      load_v(tile);
      for (int j = s0; j < s1; j++) {
        const int no = step_no + j - s0, st = no & 1;
        const uint32_t empty = ((no >> 1) & 1) ^ 1;
        const int first = tile ? walk.it.span.tile(j * kStep + sub) * 16 : -16;
        const bool sees = tile && kvp_sees_all(a, walk.it.span.p0, walk.it.span.p1, first, 16);
        // a token that no row sees may hold anything: it counts as zeros
        const bool live = sees || (tile && kvp_some_sees(a, walk.it.span.p0, walk.it.span.p1, first + tt));
        const uint8_t* next = tile_of(page_next, j + 1);
        page_next = entry(j + 2);
        mbar_wait(&ctl.k_empty[st], empty, &ctl.gave_up);
        if (tt == 0 && g0 == 0) ctl.place[no & (kRing - 1)][sub] = first | (sees ? 1 : 0);
        {
          const uint32_t z[2] = {live ? kz.x : 0u, live ? kz.y : 0u};
#pragma unroll
          for (int g = 0; g < H; g++)
            put(smem + C::kK + st * C::kTileBytes, g, kc[g], __low2half2(as_h2(z[g])), __high2half2(as_h2(z[g])));
        }
        fence_async_smem();
        mbar_arrive(&ctl.k_full[st]);
        load_k(next);
        mbar_wait(&ctl.v_empty[st], empty, &ctl.gave_up);
        {
          const uint32_t z[4] = {live ? vz.x : 0u, live ? vz.y : 0u, live ? vz.z : 0u, live ? vz.w : 0u};
#pragma unroll
          for (int g = 0; g < H; g++) {
            const __half2 ss = as_h2(z[2 * g]), mm = as_h2(z[2 * g + 1]);
            put(smem + C::kV + st * C::kTileBytes, g, vc[g], tt & 1 ? __high2half2(ss) : __low2half2(ss),
                tt & 1 ? __high2half2(mm) : __low2half2(mm));
          }
        }
        fence_async_smem();
        mbar_arrive(&ctl.v_full[st]);
        load_v(next);
        tile = next;
      }
      step_no += s1 - s0;
    } while (advance());
  } else {
    regs_down<kIssueRegs>();
    // ======================= the products =====================================
    if (warp == kSoftWarps + kFillWarps) {
      constexpr uint32_t kS = mma_desc(kTokens, false), kO = mma_desc(D, true);
      const uint32_t q_lo = desc_lo(smem_at + C::kQ, 16), k_lo0 = desc_lo(smem_at + C::kK, 16),
                     v_lo0 = desc_lo(smem_at + C::kV, 16384);
      uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0}, no = 0;  // phases of q_full, p_full; steps so far
      if (walk.s0 < walk.s1) do {
        const int steps = walk.s1 - walk.s0;
        const int tiles = walk.it.seq.n * a.group - walk.it.rt * kRows > kTileRows ? 2 : 1;
        for (int j = 0; j <= steps; j++, no++) {
          const uint32_t st = no & 1, bst = st ^ 1;  // stages of this step and of the one before
          if (j < steps) mbar_wait(&ctl.k_full[st], no >> 1 & 1, &ctl.gave_up);
          if (j > 0) mbar_wait(&ctl.v_full[bst], (no - 1) >> 1 & 1, &ctl.gave_up);
#pragma unroll
          for (int t = 0; t < 2; t++) {  // the tiles in turn: one's products run while the other's weights are made
            if (t == tiles) break;
            const uint32_t s_at = tmem + t * 128, o_at = tmem + 256 + t * D;
            if (j > 0) {  // O += P V of the step before
              mbar_wait(&ctl.p_full[t], n_p[t]++ & 1, &ctl.gave_up);
              tc_after();
              const uint32_t v_lo = v_lo0 + bst * (C::kTileBytes >> 4);
              if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kTokens / 16; ks++)
                  tc_mma_ts(o_at, s_at + ks * 8, v_lo + ks * (2048 >> 4), kDescHi, kO, ks > 0 || j > 1);
                if (t == tiles - 1) tc_commit(&ctl.v_empty[bst]);
                if (j == steps) tc_commit(&ctl.o_done[t]);
              }
              __syncwarp();
            }
            if (j < steps) {  // S = Q K, over the weights that the product before has read
              if (j == 0) mbar_wait(&ctl.q_full[t], n_q[t]++ & 1, &ctl.gave_up);
              tc_after();
              const uint32_t k_lo = k_lo0 + st * (C::kTileBytes >> 4), ql = q_lo + t * (C::kTileBytes >> 4);
              if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++) {
                  const uint32_t off = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                  tc_mma_ss(s_at, ql + off, k_lo + off, kDescHi, kDescHi, kS, ks > 0);
                }
                tc_commit(&ctl.s_full[t]);
                if (t == tiles - 1) tc_commit(&ctl.k_empty[st]);
              }
              __syncwarp();
            }
          }
        }
        no--;  // the last pass made no step
      } while (advance());
      if (elect_one()) tc_commit(&ctl.last);  // nothing is in flight when TMEM is given back
      __syncwarp();
      mbar_drain(&ctl.last, 0, &g_wait_timeouts);
    }
  }
  tc_before();
  __syncthreads();
  if (warp == kSoftWarps + kFillWarps) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// One CTA per (item, 4 or 8 rows): joins the parts of the item, in the order of
// the CTAs; 4 elements per thread.
constexpr int kMergeThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) kvp_prefill_merge_kernel(const __grid_constant__ PrefillArgs pa) {
  using C = Cfg<D>;
  constexpr int kPer = kMergeThreads / (D / 4);
  const KvpAttendArgs& a = pa.a;
  pdl_trigger();
  pdl_wait();
  const KvpShared d = pa.desc[blockIdx.x];
  const int r = blockIdx.y * kPer + threadIdx.x / (D / 4), d4 = threadIdx.x % (D / 4) * 4;
  if (d.parts == 0 || r >= d.rows) return;
  auto part = [&](int i) {  // the first lies in the starting CTA's second place, the others in their CTA's first
    return pa.parts + (size_t)(2 * (d.cta + i) + (i == 0 ? 1 : 0)) * C::kPartFloats;
  };
  float top = -INFINITY;
  for (int i = 0; i < d.parts; i++) top = fmaxf(top, part(i)[kRows * D + 2 * r]);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int i = 0; i < d.parts; i++) {
    const float* p = part(i);
    const float2 m = *reinterpret_cast<const float2*>(p + kRows * D + 2 * r);
    const float4 v = *reinterpret_cast<const float4*>(p + r * D + d4);
    const float f = m.x == -INFINITY ? 0.f : ex2(m.x - top);
    sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
    sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
    l = fmaf(f, m.y, l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int qi = kvp_by_group(a, d.row0 + r), h = d.head0 + d.row0 + r - qi * a.group;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + ((size_t)(d.q_row + qi) * a.h_q + h) * D + d4) =
      make_uint2(Elem<T>::from_float2(sum.x * inv, sum.y * inv), Elem<T>::from_float2(sum.z * inv, sum.w * inv));
}

template <typename T, int D>
sf_status launch_prefill(const KvpAttendArgs& a, cudaStream_t s) {
  using C = Cfg<D>;
  const int ctas = num_sms();
  PrefillArgs pa;
  pa.a = a;
  pa.desc = static_cast<KvpShared*>(a.ws);
  pa.parts = reinterpret_cast<float*>(pa.desc + ctas);
  const long each = (long)(a.n_q / a.batch) * a.group;
  const long items = (each + kRows - 1) / kRows * a.h_kv * a.batch;
  pa.by_item = !a.cu_q && items < ctas;
  const int entries = pa.by_item ? (int)items : ctas;
  const int most = a.cu_q ? kRows : (int)(each < kRows ? each : kRows), per = kMergeThreads / (D / 4);
  SF_CUDA((kvp_allow_smem<kvp_prefill_kernel<T, D>>(C::kSmem)));
  SF_CUDA(launch_pdl(kvp_prefill_kernel<T, D>, dim3(ctas), dim3(kThreads), C::kSmem, s, pa));
  SF_CUDA(launch_pdl(kvp_prefill_merge_kernel<T, D>, dim3(entries, (most + per - 1) / per), dim3(kMergeThreads), 0, s,
                     pa));
  return SF_OK;
}

}  // namespace

size_t kvp_prefill_workspace(int d) {
  return (size_t)num_sms() * (sizeof(KvpShared) + 2 * (kRows * d + 2 * kRows) * sizeof(float));
}

sf_status launch_kvp_prefill(const KvpAttendArgs& a, int d, sf_dtype dtype, cudaStream_t s) {
  if (d == 128) return dtype == SF_F16 ? launch_prefill<__half, 128>(a, s) : launch_prefill<__nv_bfloat16, 128>(a, s);
  return dtype == SF_F16 ? launch_prefill<__half, 64>(a, s) : launch_prefill<__nv_bfloat16, 64>(a, s);
}

cudaError_t kvp_wait_timeouts(unsigned int* count, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(unsigned int));
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(unsigned int));
  }
  return e;
}

}  // namespace sf
