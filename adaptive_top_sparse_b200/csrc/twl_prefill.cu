// Attention of prompt chunks: the last q_len tokens of every sequence attend causally over a
// sliding window and the first (sink) tokens of the sequence's paged fp16 cache.
//
// Query row i of a chunk sits at position t = n - q_len + i and sees key j iff j <= t and
// (j < sinks or j > t - window).  o = softmax(scale q K^T) V over the seen keys in one pass: the
// running maximum and sum of each row rescale the accumulator when the maximum grows.
//
// Units: the G heads of a kv-head share its keys, so a row is a (query, head) pair and a unit is
// 256 rows (256 / G queries) of one (sequence, kv-head): two query tiles of 128 rows that share
// every key tile of 128 tokens (8 pages).  The key tiles of all units form one flat list that is
// cut into equal runs, one per CTA (one CTA per SM); a unit cut by runs leaves fp32 partials that
// the CTA arriving last merges in run order.  So a few long sequences with a handful of queries
// use the card as well as one long prompt, and lengths stay on the device.
//
// One CTA: twenty warps.
//   loader     TMA of the queries and of K and V pages (a copy per page, 128-byte swizzle) into a
//              ring of five 32 KB buffers
//   fixers     two warps that zero the V rows nobody in the unit sees: a weight of 0 times a stale
//              infinity would be NaN.  A value that is not finite, in a row that only some of the
//              queries see, is zeroed too and noted, and the queries that see it get their NaN at
//              the end.  Only tiles at the edge of what is seen need either
//   mma        one thread: S_x = Q_x K^T (tcgen05, fp16 in, fp32 in TMEM) and O_x += P_x V with P
//              in TMEM over S and V taken as it lies in the page (MN-major)
//   softmax x  eight warps per query tile, two threads per row: scores from TMEM, maximum, weights
//              back to TMEM as fp16, sums in fp32.  While one tile's softmax runs, the tensor core
//              works for the other.
// The weights enter the product as fp16 (2^-11 of each, as the fp16 result itself); maxima, sums
// and accumulators are fp32.  Waits are bounded: one that gives up raises TWL_FLAG_TIMEOUT and
// the CTA leaves without its outputs.
//
// Measured (one B200, 32/8 heads; replays of a graph in short bursts, and in brackets passes back to
// back): a prompt of 8192 under a window of 2048 in 327 (357) us (736, 675 TFLOP/s), four chunks of
// 1.5K-2K over 2K-8K cached tokens in 607 (691) us (912, 801 TFLOP/s, 56 and 49 % of the measured bf16
// rate; the power cap takes part of it), 1-8 drafted tokens behind eight contexts in 44 us (3.0 TB/s).
// Bound: the chain of a query tile (some 2100 cycles of softmax, 1100 of products, and the hand-overs)
// is longer than the other tile's 1072 cycles of the tensor core.  TMEM has no room for a third tile
// of scores; the softmax has 96 registers a thread (640 equal threads), so it reads each score from
// TMEM twice, and the halves of a row meet through shared memory in every tile.
#include <cuda.h>

#include "twl_common.cuh"
#include "twl_kernels.h"
#include "twl_prefill.h"

namespace twl {
namespace prefill {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.f;  // log2: a row's maximum is raised only when exceeded by more
// Up to here a score is scaled and its maximum taken off in one fma.  The maximum is rounded, so all
// weights of a row share a factor of up to 2^(2^-24 kFar): nothing that o or lse sees.  Beyond, that
// factor would pass fp16's range: there scores in TMEM are first scaled, rounded as their maximum
// is, brought to it and scaled back.
constexpr float kFar = 0x1p20f;
constexpr int kRows = 256, kTileRows = 128, kKeys = 128;
constexpr int kThreads = 640;
constexpr int kBufBytes = 32768, kBufs = 5;
constexpr int kQBytes = 65536;
// What a unit costs beside its key tiles (filling and emptying the pipeline, masks, the output), in
// tiles: places in the flat list that hold no work, so that a run of many short units is shorter.
// Measured with 0, 1, 2 and 3 (us, 32/8 heads but for the last two): 8 x 1-8 tokens behind 2-8K under
// 4096 42.5, 41.3, 41.5, 41.6; prompt of 8K under 2048 328, 306, 306, 306; four chunks of 1.5-2K over
// 2-8K 570, 544, 545, 544; 32 chunks of 64 behind 1-4K 138, 144, 138, 138; 64 prompts of 16-400 156,
// 167, 169, 169; 1K, 64/8 heads, 65, 68, 68, 68; 16K, 8/1 heads, 662, 580, 574, 577.
constexpr int kUnitCost = 2;
constexpr int kRecs = 8;
constexpr int kSpoils = 16, kSpoilsPer = 4;  // of the CTA's last segments; of one (two a fixer)
constexpr int kMmaWarp = 16, kLoadWarp = 17, kFixWarp = 18;
// partial of a cut unit: o as [32][256] float4 (column group, row), then max[256], sum[256]
constexpr int kPartFloats = kRows * 130;

// A value of V that is not finite, in a row that some of a unit's queries see and others do not.
struct Spoil {
  int seg, key;       // the CTA's segment; the row's position
  uint32_t cols[4];   // its columns that are not finite
};

struct Smem {
  // barriers
  uint64_t q_full, q_free;
  uint64_t full[kBufs], empty[kBufs];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_free[2];
  uint64_t drain;           // the CTA's products in flight at its end
  uint64_t v_ready[kBufs];  // V of the buffer is loaded and its unseen rows are zero
  uint32_t tmem;
  uint32_t wait_limit;
  int aborted;
  int rec[kRecs];  // of a key tile: pages that were loaded (bit per page), its number << 8
  int is_last;
  uint32_t spoils;        // whether any segment so far has one
  Spoil spoil[kSpoils];   // segment s: at kSpoilsPer (s % 4)
  // where the run starts
  int b, kvh, qt, tile;
  float swap[2][2][kTileRows];  // maxima and sums of the halves of the rows
};
constexpr size_t kSmemBytes = kQBytes + (size_t)kBufs * kBufBytes + sizeof(Smem);

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t sptr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sptr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sptr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(sptr(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(sptr(b)), "r"(parity), "r"(20000u) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_try_now(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(sptr(b)), "r"(parity) : "memory");
  return ok != 0;
}
constexpr uint32_t kWaitLimit = 1u << 16;  // polls of up to 20 us each (Args.wait_limit)
// An arrival at a cut unit's counter; one of a run that gave up counts in the upper half too.
constexpr unsigned kArrived = 1u, kGaveUp = 0x10000u;

// Waits for the phase of the given parity; false when the wait, or another in the CTA, gave up.
__device__ __forceinline__ bool bar_wait(Smem& s, uint64_t* b, uint32_t parity, uint32_t* flags) {
  for (uint32_t i = 0; i < s.wait_limit; ++i) {
    if (bar_try(b, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&s.aborted)) return false;
  }
  *reinterpret_cast<volatile int*>(&s.aborted) = 1;
  raise_flag(flags, TWL_FLAG_TIMEOUT);
  return false;
}
// The same for a converged warp, with one answer for all of its lanes.
__device__ __forceinline__ bool warp_wait(Smem& s, uint64_t* b, uint32_t parity, uint32_t* flags) {
  if (__all_sync(0xffffffffu, bar_try_now(b, parity))) return true;
  return __all_sync(0xffffffffu, bar_wait(s, b, parity, flags));
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// A page of one kv-head, coordinate y = its first row / 8: see the maps in launch_g.
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int y,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(0), "r"(y), "r"(sptr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(sptr(bar))
      : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: lead and stride are the distances in bytes
// between 64-element blocks of the contiguous dimension (MN-major only) and between groups of 8
// rows of the other one.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(stride >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor: fp16 x fp16 -> fp32, M = 128, N = 128; B as K-major or MN-major.
constexpr uint32_t kIdescQK = 1u << 4 | (128u / 8) << 17 | (128u / 16) << 24;
constexpr uint32_t kIdescPV = kIdescQK | 1u << 16;

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
      "r"(kIdescQK), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b),
      "r"(kIdescPV), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sptr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define TWL_R8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), \
                     "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
#define TWL_O8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                     "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define TWL_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                     "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of the warp's 32 lanes: register c of lane l = column c of TMEM lane l.  The values
// are there after wait_ld (keep_ld ties them to it).
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : TWL_O8(r, 0), TWL_O8(r, 8), TWL_O8(r, 16), TWL_O8(r, 24) : "r"(addr));
}
__device__ __forceinline__ void keep_ld(uint32_t (&r)[32]) {
  asm volatile("" : TWL_R8(r, 0), TWL_R8(r, 8), TWL_R8(r, 16), TWL_R8(r, 24));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(addr),
      TWL_I8(r, 0), TWL_I8(r, 8), TWL_I8(r, 16), TWL_I8(r, 24) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];" : TWL_O8(r, 0), TWL_O8(r, 8) : "r"(addr));
}
__device__ __forceinline__ void keep_ld16(uint32_t (&r)[16]) {
  asm volatile("" : TWL_R8(r, 0), TWL_R8(r, 8));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr), TWL_I8(r, 0), TWL_I8(r, 8) : "memory");
}

// 32 bytes, a whole sector (the rows of a warp's lanes are far apart).
__device__ __forceinline__ void st_global32(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), TWL_I8(r, 0)
               : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x without the special function unit, whose one result in 8 cycles a warp is as much of a bound
// as the tensor core: x = i + f with f in [-0.5, 0.5] by rounding through 1.5 2^23, 2^f by a
// polynomial (degree 4, fitted for the least relative error, 2.7e-6), i added to the exponent.
// Below 2^-125 the result stays there: 0 as fp16.  NaN does too: such a score reaches the row by
// its maximum (max3).
__device__ __forceinline__ float exp2_poly(float x) {
  x = fmaxf(x, -125.f);
  const float i = __fadd_rn(x, 0x1.8p23f);
  const float f = x - __fsub_rn(i, 0x1.8p23f);
  float y = fmaf(f, 0.009570102207362652f, 0.05591785907745361f);
  y = fmaf(y, f, 0.240247443318367f);
  y = fmaf(y, f, 0.6931217908859253f);
  y = fmaf(y, f, 0.9999992847442627f);
  return __uint_as_float(__float_as_uint(y) + (__float_as_uint(i) << 23));
}
// Maxima that are NaN when an operand is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max2(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Two fp32 values in one register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
  return y;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t y;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}
// Weights of 32 scores, as fp16 pairs, and their sums (two in a pair).  One in eight by polynomial:
// then the special function unit and the instruction issue are about even.
__device__ __forceinline__ void weights(const uint32_t (&v)[32], uint64_t scale, uint64_t shift,
                                        uint64_t& sum, uint32_t (&p)[16]) {
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    const uint64_t x = fma2((uint64_t)v[k + 1] << 32 | v[k], scale, shift);
    const float x0 = __uint_as_float((uint32_t)x), x1 = __uint_as_float((uint32_t)(x >> 32));
    const float p0 = exp2_fast(x0);
    const float p1 = (k & 6) == 6 ? exp2_poly(x1) : exp2_fast(x1);
    sum = add2(sum, pack2(p0, p1));
    const __half2 h = __floats2half2_rn(p0, p1);
    p[k >> 1] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
// The lowest n of 32 bits (none for n <= 0).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}
// Which of the columns c .. c + 31 of a key tile a row sees: column <= hi and (column > lo or
// column < sk), on pages that were loaded.
__device__ __forceinline__ uint32_t seen_bits(int c, int hi, int lo, int sk, int pages) {
  const uint32_t on = (pages >> (c / kPage) & 1 ? 0x0000FFFFu : 0u) |
                      (pages >> (c / kPage + 1) & 1 ? 0xFFFF0000u : 0u);
  return low_bits(hi - c + 1) & (~low_bits(lo - c + 1) | low_bits(sk - c)) & on;
}
__device__ __forceinline__ void hide(uint32_t (&v)[32], uint32_t seen) {
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = seen >> k & 1u ? v[k] : 0xFF800000u;
}
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// Brings 64 columns of scores that lie far from 0 to their row's maximum (see kFar).
__device__ __noinline__ void far_scores(uint32_t ts, float scale, float ref) {
  const float back = 1.f / scale;
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    uint32_t s[16];
    tmem_ld16(s, ts + c);
    wait_ld();
    keep_ld16(s);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      s[k] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(s[k]), scale), ref) * back);
    tmem_st16(ts + c, s);
  }
  wait_st();
}

// ------------------------------------------------------------------ the flat list
struct Chunk {
  int qs, qn, n;  // first row of q, queries, cached length
};

// Sequence b's chunk; qn = 0 (and a flag, by `report`) when it cannot be served.
__device__ __forceinline__ Chunk chunk_of(const Args& a, int b, bool report) {
  Chunk c;
  c.qs = a.q_start[b];
  const int e = a.q_start[b + 1];
  c.n = a.seq_lens[b];
  c.qn = e - c.qs;
  if (c.qs < 0 || e < c.qs || e > a.total_q || c.n < c.qn || c.n > a.max_pages * kPage) {
    if (report) raise_flag(a.flags, TWL_FLAG_BAD_INDEX);
    c.qn = 0;
  }
  return c;
}

// The keys of a unit of queries [i0, i0 + queries) of a chunk.
struct Span {
  int t0, t1;              // positions of its first and last query
  int lo;                  // first key of any of its windows
  int sink_tiles, first;   // tiles of the sinks; first tile behind them
  int tiles;
};
__device__ __forceinline__ Span span_of(const Args& a, const Chunk& c, int i0, int queries) {
  Span s;
  s.t0 = c.n - c.qn + i0;
  s.t1 = min(s.t0 + queries, c.n) - 1;
  s.lo = s.t0 >= a.window ? s.t0 - a.window + 1 : 0;
  s.first = s.lo / kKeys;
  s.sink_tiles = min((min(a.sinks, c.n) + kKeys - 1) / kKeys, s.first);
  s.tiles = s.sink_tiles + s.t1 / kKeys - s.first + 1;
  return s;
}

// Which of two fp16 values are not finite (bits 0 and 1), and the two with 0 in place of those.
__device__ __forceinline__ uint32_t odd_values(uint32_t x) {
  return ((x & 0x7C00u) == 0x7C00u ? 1u : 0u) | ((x & 0x7C000000u) == 0x7C000000u ? 2u : 0u);
}
__device__ __forceinline__ uint32_t keep_finite(uint32_t x) {
  const uint32_t b = odd_values(x);
  return (b & 1 ? 0u : x & 0xFFFFu) | (b & 2 ? 0u : x & 0xFFFF0000u);
}

// A fixer warp: zeroes what is not finite in its 64 rows of a V tile (the first at position key0)
// and notes the rows and columns for segment seg.  A warp has room for two rows of a segment;
// further ones go to its second, under the lower of their positions.
__device__ __noinline__ void spoilt_rows(Smem& s, unsigned char* v, int key0, int seg, int half) {
  const int lane = threadIdx.x & 31;
  Spoil* of = s.spoil + (seg % (kSpoils / kSpoilsPer)) * kSpoilsPer + 2 * half;
#pragma unroll 1
  for (int it = 0; it < 32; ++it) {
    // 512 bytes: 4 rows of one half of the columns, chunks of 8 columns swizzled by row
    const int r = (it >> 2) * 8 + (it & 1) * 4 + (lane >> 3);
    uint4* at = reinterpret_cast<uint4*>(v + it * 512 + lane * 16);
    const uint4 x = *at;
    const uint32_t bad = odd_values(x.x) | odd_values(x.y) << 2 | odd_values(x.z) << 4 |
                         odd_values(x.w) << 6;
    if (bad)
      *at = make_uint4(keep_finite(x.x), keep_finite(x.y), keep_finite(x.z), keep_finite(x.w));
    const int col = (it >> 1 & 1) * 64 + (((lane & 7) ^ (r & 7)) * 8);
    for (unsigned who = __ballot_sync(0xffffffffu, bad != 0); who; who &= who - 1) {
      const int l = __ffs(who) - 1;
      const uint32_t m = __shfl_sync(0xffffffffu, bad, l);
      const int c = __shfl_sync(0xffffffffu, col, l), key = key0 + __shfl_sync(0xffffffffu, r, l);
      if (lane != 0) continue;
      for (int i = 0; i < 2; ++i) {
        const bool fresh = of[i].seg != seg;
        if (fresh) {
          of[i].key = key;
          for (int w = 0; w < 4; ++w) of[i].cols[w] = 0u;
          of[i].seg = seg;
        }
        if (of[i].key == key || i == 1) {
          of[i].key = min(of[i].key, key);
          of[i].cols[c >> 5] |= m << (c & 31);
          break;
        }
      }
    }
    __syncwarp();
  }
  if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&s.spoils) = 1u;
}

// Where run i of `runs` starts in a list of `total`.
__device__ __forceinline__ long long cut_at(long long total, int i, int runs) {
  if (total < (1 << 20)) return (unsigned)total * (unsigned)i / (unsigned)runs;  // far cheaper
  return total * i / runs;
}

// The run that holds tile f.
__device__ __forceinline__ int run_of(long long f, long long total, int runs) {
  if (total < (1 << 20))
    return (int)((((unsigned)f + 1u) * (unsigned)runs - 1u) / (unsigned)total);
  return (int)(((f + 1) * runs - 1) / total);
}

// Every role walks the CTA's run of the list by itself: segments of units, in order.
template <int G>
struct Walk {
  static constexpr int kQueries = kRows / G;
  const Args* args;
  long long at, end;     // place in the flat list
  int b, kvh, qt, tile;  // of the next segment (tile: its place in the unit)
  Chunk c;
  // the current segment
  Span s;
  int i0, tile0, tiles;  // first query, first key tile, key tiles
  long long start;       // the unit's place in the list
  bool whole, two;       // the whole unit; it has rows in the second query tile

  __device__ Walk(const Args& a, const Smem& sm, long long f0, long long f1)
      : args(&a), at(f0), end(f1), b(sm.b), kvh(sm.kvh), qt(sm.qt), tile(sm.tile) {
    if (at < end) c = chunk_of(a, b, false);
  }
  __device__ bool next() {
    const Args& a = *args;
    do {
      if (at >= end) return false;
      while (qt * kQueries >= c.qn) {
        qt = 0;
        if (++kvh >= a.hkv || c.qn == 0) {
          kvh = 0;
          c = chunk_of(a, ++b, false);
        }
      }
      i0 = qt * kQueries;
      s = span_of(a, c, i0, kQueries);
      tile0 = tile;
      start = at - tile;
      const int take = (int)min((long long)(s.tiles + kUnitCost - tile), end - at);
      tiles = min(tile + take, s.tiles) - tile;
      at += take;
      tile += take;
      if (tile == s.tiles + kUnitCost) tile = 0, ++qt;
    } while (tiles <= 0);
    whole = tiles == s.tiles;
    two = i0 + kTileRows / G < c.qn;
    return true;
  }
  // First token of the segment's key tile i.
  __device__ int base_of(int i) const {
    const int x = tile0 + i;
    return (x < s.sink_tiles ? x : s.first + x - s.sink_tiles) * kKeys;
  }
  // Whether some query of the unit does not see some key of the tile at `base`.
  __device__ bool mixed(int base, int pages) const {
    return pages != 0xFF || base + kKeys - 1 > s.t0 ||
           (base <= s.t1 - args->window && base + kKeys > args->sinks);
  }
};

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_prefill(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ __align__(1024) unsigned char base_ptr[];
  unsigned char* qbuf = base_ptr;
  unsigned char* ring = base_ptr + kQBytes;
  Smem& sm = *reinterpret_cast<Smem*>(ring + (size_t)kBufs * kBufBytes);
  long long* prefix = reinterpret_cast<long long*>(ring);  // [batch + 1], before the first load
  constexpr int kQueries = kRows / G;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == kLoadWarp * 32) {
    sm.wait_limit = a.wait_limit;
    sm.aborted = 0;
    sm.spoils = 0;
    for (int i = 0; i < kSpoils; ++i) sm.spoil[i].seg = -1;
    bar_init(&sm.q_full, 1);
    bar_init(&sm.q_free, 1);
    bar_init(&sm.drain, 1);
    for (int i = 0; i < kBufs; ++i) bar_init(&sm.full[i], 1), bar_init(&sm.empty[i], 3);
    for (int x = 0; x < 2; ++x) {
      bar_init(&sm.s_full[x], 1);
      bar_init(&sm.p_half[x], 8);
      bar_init(&sm.p_full[x], 8);
      bar_init(&sm.o_full[x], 1);
      bar_init(&sm.o_free[x], 8);
    }
    for (int i = 0; i < kBufs; ++i) bar_init(&sm.v_ready[i], 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     sptr(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // ---- prefix[b] = key tiles per kv-head of the sequences before b
  for (int b = warp; b < a.batch; b += kThreads / 32) {
    const Chunk c = chunk_of(a, b, blockIdx.x == 0 && lane == 0);
    long long sum = 0;
    for (int i = lane * kQueries; i < c.qn; i += 32 * kQueries)
      sum += span_of(a, c, i, kQueries).tiles + kUnitCost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) prefix[b + 1] = sum;
  }
  if (tid == 0) prefix[0] = 0;
  __syncthreads();
  if (warp == 0) {
    long long carry = 0;
    for (int b0 = 1; b0 <= a.batch; b0 += 32) {
      long long x = b0 + lane <= a.batch ? prefix[b0 + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      x += carry;
      if (b0 + lane <= a.batch) prefix[b0 + lane] = x;
      carry = __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const long long total = prefix[a.batch] * a.hkv;
  const int runs = (int)min((long long)gridDim.x, total);
  const int run = blockIdx.x;
  if (run >= runs) {
    __syncthreads();  // the allocation is there
    if (warp == kMmaWarp)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem));
    return;
  }
  const long long f0 = cut_at(total, run, runs), f1 = cut_at(total, run + 1, runs);
  if (warp == 0) {
    int x = 0, y = a.batch;  // prefix[x] hkv <= f0 < prefix[y] hkv
    while (y - x > 1) {
      const int mid = (x + y) >> 1;
      if (prefix[mid] * a.hkv <= f0) x = mid;
      else y = mid;
    }
    const long long per = prefix[x + 1] - prefix[x], in = f0 - prefix[x] * a.hkv;
    long long rest = in % per;
    const Chunk c = chunk_of(a, x, false);
    for (int q0 = 0;; q0 += 32) {  // the unit that holds tile `rest` of this kv-head
      const int i = (q0 + lane) * kQueries;
      const int t = i < c.qn ? span_of(a, c, i, kQueries).tiles + kUnitCost : 0;
      int sum = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, rest < sum);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          sm.b = x;
          sm.kvh = (int)(in / per);
          sm.qt = q0 + lane;
          sm.tile = (int)(rest - (sum - t));
        }
        break;
      }
      rest -= __shfl_sync(0xffffffffu, sum, 31);
      if (q0 * kQueries >= c.qn) break;  // not reached: rest is below the sum of all units
    }
  }
  fence_before();
  // the prefix lay where TMA writes next
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  Walk<G> w(a, sm, f0, f1);
  auto dead = [&]() { return *reinterpret_cast<volatile int*>(&sm.aborted) != 0; };

  if (warp == kLoadWarp) {
    // ================================================================ loader
    int fill = 0, ntile = 0, nseg = 0;
    bool ok = true;
    while (ok && w.next()) {
      if (nseg > 0) ok = warp_wait(sm, &sm.q_free, (nseg - 1) & 1, a.flags);
      if (!ok) break;
      ++nseg;
      if (lane == 0) {
        bar_expect(&sm.q_full, w.two ? kQBytes : kQBytes / 2);
        for (int x = 0; x < (w.two ? 2 : 1); ++x)
          for (int h = 0; h < 2; ++h)
            tma_3d(sptr(qbuf) + x * 32768 + h * 16384, &qmap, 64 * h, w.kvh * G,
                   w.c.qs + w.i0 + x * (kTileRows / G), &sm.q_full);
      }
      for (int i = 0; i < w.tiles; ++i, ++ntile) {
        const int base = w.base_of(i);
        int phys = -1;
        if (lane < kKeys / kPage) {
          const int p0 = base + lane * kPage;
          if (p0 <= w.s.t1 && (p0 < a.sinks || p0 + kPage > w.s.lo))
            phys = load_phys(a.page_table, w.b, p0 / kPage, a.max_pages, a.num_phys, a.flags);
        }
        const unsigned pages = __ballot_sync(0xffffffffu, phys >= 0);
        for (int kv = 0; kv < 2; ++kv, ++fill) {
          const int buf = fill % kBufs, round = fill / kBufs;
          if (round > 0 && !warp_wait(sm, &sm.empty[buf], (round - 1) & 1, a.flags)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (kv == 0) sm.rec[ntile % kRecs] = (int)pages | (base / kKeys) << 8;
            bar_expect(&sm.full[buf], __popc(pages) * 4096);
          }
          __syncwarp();
          if (phys >= 0)
            tma_page(sptr(ring) + buf * kBufBytes + lane * 4096, kv == 0 ? &kmap : &vmap,
                     (phys * a.hkv + w.kvh) * (kPage / 8), &sm.full[buf]);
        }
        if (!ok) break;
      }
    }
    // the CTA leaves only behind its copies in flight, whoever gave up and when
    const long long t0 = clock64();
    for (int k = max(0, fill - kBufs); k < fill; ++k)
      while (!bar_try(&sm.full[k % kBufs], (k / kBufs) & 1) && clock64() - t0 < 2000000000ll) {
      }
    if (nseg > 0)
      while (!bar_try(&sm.q_full, (nseg - 1) & 1) && clock64() - t0 < 2000000000ll) {
      }
  } else if (warp == kMmaWarp) {
    // ================================================================ tensor core
    // One thread walks, waits and issues.  What it does between two products is time the tensor
    // core may idle, so ring places and phases are kept as running values (no division), and
    // everything a product needs but its weights has been waited for while the product before it ran.
    if (lane == 0) {
      bool ok = true;
      uint32_t full_ph = 0, ready_ph = 0, p_ph = 0, free_ph = 0, q_ph = 0;
      int kb = 0, units[2] = {0, 0};  // buffer of the next K
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!bar_try_now(bar, parity)) ok = ok && bar_wait(sm, bar, parity, a.flags);
      };
      auto next_buf = [](int b) { return b + 1 == kBufs ? 0 : b + 1; };
      auto wait_k = [&](int b) {
        wait(&sm.full[b], full_ph >> b & 1);
        full_ph ^= 1u << b;
      };
      auto wait_v = [&](int b) {  // a buffer takes K and V in turn
        wait(&sm.v_ready[b], ready_ph >> b & 1);
        ready_ph ^= 1u << b;
        full_ph ^= 1u << b;
      };
      // key tiles: 16 groups of 8 rows, the two 64-column halves of a group behind one another
      const uint64_t dq = smem_desc(sptr(qbuf), 16, 1024), dk = smem_desc(sptr(ring), 16, 2048),
                     dv = smem_desc(sptr(ring), 1024, 2048);
      auto scores = [&](int x, int b, bool second) {
        const uint64_t a0 = dq + (second ? 32768u >> 4 : 0u),
                       b0 = dk + (uint64_t)(b * (kBufBytes >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t in = (k & 3) * (32 >> 4);
          mma_ss(tmem + x * 128, a0 + (k >> 2) * (16384 >> 4) + in,
                 b0 + (k >> 2) * (1024 >> 4) + in, k > 0);
        }
        mma_commit(&sm.s_full[x]);
      };
      auto product = [&](int x, int vb, bool first) {  // O_x += P_x V, waits for the weights
        if (first && units[x] > 0) {
          wait(&sm.o_free[x], free_ph >> x & 1);
          free_ph ^= 1u << x;
        }
        const uint64_t v0 = dv + (uint64_t)(vb * (kBufBytes >> 4));
        const uint32_t ph = p_ph >> x & 1;
        p_ph ^= 1u << x;
        // half of the weights come first: columns 0 .. 31 and 64 .. 95 (those of columns 64 .. lie
        // over those columns' scores)
        wait(&sm.p_half[x], ph);
        if (!ok) return;
        fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int ks = (k & 1) + (k >> 1 & 1) * 4 + (k >> 2) * 2;  // 0 1 4 5, 2 3 6 7
          if (k == 4) {
            wait(&sm.p_full[x], ph);
            if (!ok) return;
            fence_after();
          }
          mma_ts(tmem + 256 + x * 128, tmem + x * 128 + (ks >> 2) * 64 + (ks & 3) * 8,
                 v0 + ks * (4096 >> 4), !first || k > 0);
        }
      };
      auto first_scores = [&](int b) {  // of a unit, for side 0
        wait(&sm.q_full, q_ph);
        q_ph ^= 1;
        wait_k(b);
        if (!ok) return;
        fence_after();
        scores(0, b, false);
      };
      Walk<G> ahead = w;
      bool more = w.next(), begun = false;
      // (a test of the waits makes every second run wait for products that nothing issues)
      if (a.stall && (run & 1)) wait(&sm.drain, 0);
      while (ok && more) {
        if (!begun) first_scores(kb);
        if (!ok) break;
        begun = false;
        ahead = w;
        more = ahead.next();
        if (w.two) {
          // two query tiles, every key tile for both
          scores(1, kb, true);
          mma_commit(&sm.empty[kb]);
          if (w.tiles == 1) mma_commit(&sm.q_free);
          wait_v(next_buf(kb));
          for (int i = w.tiles; i > 0 && ok; --i) {
            const int vb = next_buf(kb), kn = next_buf(vb);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              product(x, vb, i == w.tiles);
              if (!ok) break;
              if (x == 1) mma_commit(&sm.empty[vb]);
              if (i == 1) {
                mma_commit(&sm.o_full[x]);
                ++units[x];
                if (x == 0 && more && ahead.two) {
                  // the next unit's first scores, while side 1 of this one finishes
                  first_scores(kn);
                  begun = true;
                  if (!ok) break;
                }
              } else {
                if (x == 0) wait_k(kn);
                else wait_v(next_buf(kn));
                if (!ok) break;
                scores(x, kn, x == 1);
              }
            }
            if (!ok) break;
            if (i > 1) mma_commit(&sm.empty[kn]);
            if (i == 2) mma_commit(&sm.q_free);
            kb = kn;
          }
        } else {
          // one query tile: even key tiles go through side 0 of TMEM, odd ones through side 1
          mma_commit(&sm.empty[kb]);
          if (w.tiles > 1) {
            const int k1 = next_buf(next_buf(kb));
            wait_k(k1);
            if (!ok) break;
            scores(1, k1, false);
            mma_commit(&sm.empty[k1]);
          }
          if (w.tiles <= 2) mma_commit(&sm.q_free);
          for (int j = 0; j < w.tiles && ok; ++j) {
            const int x = j & 1, vb = next_buf(kb), kn = next_buf(vb);
            wait_v(vb);
            product(x, vb, j < 2);
            if (!ok) break;
            mma_commit(&sm.empty[vb]);
            if (j + 2 >= w.tiles) {
              mma_commit(&sm.o_full[x]);
              ++units[x];
            } else {
              const int k2 = next_buf(next_buf(kn));
              wait_k(k2);
              if (!ok) break;
              scores(x, k2, false);
              mma_commit(&sm.empty[k2]);
              if (j + 3 == w.tiles) mma_commit(&sm.q_free);
            }
            kb = kn;
          }
        }
        w = ahead;
      }
      // the CTA gives TMEM back only behind its products, whoever gave up and when
      mma_commit(&sm.drain);
      const long long t0 = clock64();
      while (!bar_try(&sm.drain, 0) && clock64() - t0 < 2000000000ll) {
      }
    }
    __syncwarp();
  } else if (warp >= kFixWarp) {
    // ================================================================ fixers
    int fill = 0, ntile = 0, seg = -1;
    bool ok = true;
    while (ok && w.next()) {
      ++seg;
      for (int i = 0; i < w.tiles && ok; ++i, ++ntile) {
        for (int kv = 0; kv < 2; ++kv, ++fill) {
          const int buf = fill % kBufs;
          ok = warp_wait(sm, &sm.full[buf], (fill / kBufs) & 1, a.flags);
          if (!ok) break;
          const int rec = sm.rec[ntile % kRecs], base = (rec >> 8) * kKeys, pages = rec & 0xFF;
          if (kv == 1 && w.mixed(base, pages)) {
            // this warp's 64 rows: 8 groups of 8 rows, 2 KB each
            const int half = warp - kFixWarp;
            unsigned char* v = ring + buf * kBufBytes + half * (kBufBytes / 2);
            for (int r = lane; r < 64; r += 32) {
              const int key = base + half * 64 + r;
              const bool seen = key <= w.s.t1 && (key < a.sinks || key >= w.s.lo) &&
                                (pages >> ((half * 64 + r) / kPage) & 1);
              if (!seen) {
                unsigned char* p = v + (r >> 3) * 2048 + (r & 7) * 128;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const int cc = ((c + lane) & 7) * 16;
                  *reinterpret_cast<uint4*>(p + cc) = make_uint4(0, 0, 0, 0);
                  *reinterpret_cast<uint4*>(p + 1024 + cc) = make_uint4(0, 0, 0, 0);
                }
              }
            }
            __syncwarp();
            uint32_t bad = 0;  // an exponent of all ones carries into the bit above it
#pragma unroll 8
            for (int it = 0; it < 32; ++it) {
              const uint4 x = *reinterpret_cast<const uint4*>(v + it * 512 + lane * 16);
              bad |= ((x.x & 0x7C007C00u) + 0x04000400u) | ((x.y & 0x7C007C00u) + 0x04000400u) |
                     ((x.z & 0x7C007C00u) + 0x04000400u) | ((x.w & 0x7C007C00u) + 0x04000400u);
            }
            if (__any_sync(0xffffffffu, (bad & 0x80008000u) != 0))
              spoilt_rows(sm, v, base + half * 64, seg, half);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) {
            if (kv == 1) bar_arrive(&sm.v_ready[buf]);
            bar_arrive(&sm.empty[buf]);
          }
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ================================================================ softmax of query tile x
    // Two threads per row: columns 64 half .. of the scores, dims 64 half .. of the output.
    const int x = warp >> 3, half = warp >> 2 & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + lanes + x * 128 + half * 64;
    const uint32_t to = tmem + lanes + 256 + x * 128 + half * 64;
    const int pair_bar = 2 + x * 4 + (warp & 3);
    float* mine = &sm.swap[x][half][row];
    const float* other = &sm.swap[x][half ^ 1][row];
    uint32_t sph = 0, oph = 0;
    int seg = -1;
    uint32_t ntile = 0;  // key tiles so far, of the CTA
    while (w.next()) {
      ++seg;
      // one query tile: side x of TMEM has every second key tile of the same rows
      const int xq = w.two ? x : 0, step = w.two ? 1 : 2, first_tile = w.two ? 0 : x;
      const int i = w.i0 + (xq * kTileRows + row) / G;  // the row's query
      const int t = w.c.n - w.c.qn + i;
      const bool active = first_tile < w.tiles;
      const bool valid = i < w.c.qn;
      float m = -INFINITY, l = 0.f;
      // first and last query of this tile of rows: tiles of keys that all of them see need no mask
      const int ta = w.s.t0 + xq * (kTileRows / G), tb = min(ta + kTileRows / G, w.c.n) - 1;
      for (int j = first_tile; j < w.tiles; j += step) {
        const bool live = warp_wait(sm, &sm.s_full[x], sph, a.flags);
        sph ^= 1;
        fence_after();
        const int rec = sm.rec[(ntile + j) % kRecs], base = (rec >> 8) * kKeys, pages = rec & 0xFF;
        const bool clear = pages == 0xFF && base + kKeys - 1 <= ta &&
                           (base > tb - a.window || base + kKeys <= a.sinks);
        // The columns are read twice, for their maximum and for their weights, and the weights'
        // loop is kept short: with the row unrolled, half of the softmax warps' time went to
        // fetching instructions.
        float m0 = -INFINITY, m1 = -INFINITY;
        int dark = 0;
        if (clear) {
          uint32_t v0[32], v1[32];
          tmem_ld32(v0, ts);
          tmem_ld32(v1, ts + 32);
          wait_ld();
          keep_ld(v0);
          keep_ld(v1);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            m0 = max3(m0, __uint_as_float(v0[k]), __uint_as_float(v0[k + 1]));
            m1 = max3(m1, __uint_as_float(v1[k]), __uint_as_float(v1[k + 1]));
          }
        } else if (live) {
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            uint32_t v[32];
            tmem_ld32(v, ts + c);
            wait_ld();
            keep_ld(v);
            // hidden scores become -inf here, in TMEM too; columns no row of the warp sees are
            // skipped from here on
            const uint32_t seen = seen_bits(half * 64 + c, t - base, max(t - a.window, -1) - base,
                                            a.sinks - base, pages);
            if (!__any_sync(0xffffffffu, seen != 0)) {
              dark |= 1 << (c / 32);
              continue;
            }
            hide(v, seen);
            tmem_st32(ts + c, v);
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              m0 = max3(m0, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
              m1 = max3(m1, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
            }
          }
          wait_st();
        }
        m0 = max2(m0, m1);
        // the halves agree on the row's maximum (they write the next one only behind the next
        // scores, which need both of them)
        *mine = m0;
        uint32_t v[32];
        tmem_ld32(v, ts);  // the first columns again, under way while the halves meet
        named_sync(pair_bar, 64);
        if (!live) {
          wait_ld();
          continue;
        }
        const float top = max2(m0, *other) * a.scale_log2;
        // (a difference: of two large numbers it is exact, and of two -inf NaN, a raise to -inf)
        if (__any_sync(0xffffffffu, !(top - m <= kSlack))) {
          // a row that has seen a score of NaN or +inf is NaN from here on: sum, lse and all of o
          float mn = max2(m, top);
          if (mn == INFINITY) mn = NAN;
          const float f = exp2_fast(m - ref_of(mn));
          m = mn;
          l *= f;
          if (j != first_tile) {  // this tile's scores were issued behind the last product into O
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
              uint32_t o[16];
              tmem_ld16(o, to + c);
              wait_ld();
              keep_ld16(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(to + c, o);
            }
          }
        }
        const float ref = ref_of(m);
        float shift = -ref;
        if (__any_sync(0xffffffffu, fabsf(ref) > kFar)) {
          wait_ld();
          far_scores(ts, a.scale_log2, ref);  // (inline it takes 2 % of a prompt, called nothing)
          tmem_ld32(v, ts);
          shift = 0.f;
        }
        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), shift2 = pack2(shift, shift);
        uint64_t sum = 0;
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          uint32_t p[16];
          wait_ld();
          keep_ld(v);
          if (dark >> (c / 32) & 1) {
#pragma unroll
            for (int k = 0; k < 16; ++k) p[k] = 0u;
          } else {
            weights(v, scale2, shift2, sum, p);
          }
          if (c == 0) tmem_ld32(v, ts + 32);
          // the weights' columns lie over scores of this thread that have been read by now
          tmem_st16(ts + (c >> 1), p);
          if (c == 0) {
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&sm.p_half[x]);
          }
        }
        l += __uint_as_float((uint32_t)sum) + __uint_as_float((uint32_t)(sum >> 32));
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.p_full[x]);
      }
      ntile += w.tiles;
      // ---- the unit's rows
      named_sync(pair_bar, 64);  // the other half has read the last maximum
      *mine = l;
      named_sync(pair_bar, 64);
      l += *other;
      named_sync(pair_bar, 64);
      if (active && warp_wait(sm, &sm.o_full[x], oph, a.flags)) fence_after();
      if (active) oph ^= 1;
      const bool fine = !__any_sync(0xffffffffu, dead());
      const size_t out = (size_t)(w.c.qs + i) * a.hq + w.kvh * G + row % G;
      float* part = a.part + ((size_t)run * 2 + (w.tile0 > 0 ? 0 : 1)) * kPartFloats;
      const int prow = x * kTileRows + row;
      const bool direct = w.whole && (w.two || w.tiles == 1);  // nothing to merge
      if (active && fine) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t o[32];
          tmem_ld32(o, to + 32 * c);
          wait_ld();
          keep_ld(o);
          if (*reinterpret_cast<volatile uint32_t*>(&sm.spoils) != 0) {
            for (int e = 0; e < kSpoils; ++e) {
              const Spoil& sp = sm.spoil[e];
              if (sp.seg != seg || sp.key > t || (sp.key >= a.sinks && sp.key <= t - a.window))
                continue;
              const uint32_t cols = sp.cols[half * 2 + c];
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = cols >> k & 1u ? 0x7FC00000u : o[k];
            }
          }
          if (valid && direct) {
            uint32_t h[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const __half2 v = __floats2half2_rn(__uint_as_float(o[k]) * inv,
                                                  __uint_as_float(o[k + 1]) * inv);
              h[k >> 1] = *reinterpret_cast<const uint32_t*>(&v);
            }
            uint16_t* dst = a.o + out * kHeadDim + 64 * half + 32 * c;
            st_global32(dst, h);
            st_global32(dst + 16, h + 8);
          } else if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(part);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[(16 * half + 8 * c + k) * kRows + prow] =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          __syncwarp();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.o_free[x]);
        if (valid && direct && half == 0)
          a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      if (direct) continue;
      if (valid && half == 0) {  // a side without a tile has seen nothing
        part[kRows * kHeadDim + prow] = active ? m : -INFINITY;
        part[kRows * (kHeadDim + 1) + prow] = active ? l : 0.f;
      }
      // ---- a cut unit: the run that arrives last merges the partials, in run order
      const int first = run_of(w.start, total, runs),
                last = run_of(w.start + w.s.tiles - 1, total, runs);
      __threadfence();
      named_sync(1, 512);
      // A run that gave up arrives too, so that the counter is zero again for the next launch; the
      // rows of its units are not written.
      if (tid == 0) {
        bool merge = !dead();
        if (first != last) {
          const unsigned before = atomicAdd(a.done + first, merge ? kArrived : kArrived + kGaveUp);
          const bool all = (before & (kGaveUp - 1)) == (unsigned)(last - first);
          if (all) a.done[first] = 0u;
          merge = merge && all && before < kGaveUp;
        }
        sm.is_last = merge;
      }
      named_sync(1, 512);
      if (sm.is_last) {
        __threadfence();
        const int rows = min(kRows, (w.c.qn - w.i0) * G);
        const int sides = w.two ? 1 : 2;  // partials of a row in each run
        auto at = [&](int k) {  // the unit starts in run `first`: its second slot
          const int r = first + (k >> (sides - 1));
          return a.part + ((size_t)r * 2 + (r == first ? 1 : 0)) * kPartFloats +
                 (k & (sides - 1)) * kTileRows;
        };
        auto o_at = [&](int k) {
          const int r = first + (k >> (sides - 1));
          return reinterpret_cast<const float4*>(
                     a.part + ((size_t)r * 2 + (r == first ? 1 : 0)) * kPartFloats) +
                 (k & (sides - 1)) * kTileRows;
        };
        const int parts = (last - first + 1) * sides;
        for (int e = tid; e < rows * 32; e += 512) {
          const int r = e % rows, c = e / rows;
          float mm = -INFINITY;
#pragma unroll 4
          for (int k = 0; k < parts; ++k) mm = fmaxf(mm, __ldcg(at(k) + kRows * kHeadDim + r));
          const float ref = ref_of(mm);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          float ll = 0.f;
#pragma unroll 4
          for (int k = 0; k < parts; ++k) {
            const float mk = __ldcg(at(k) + kRows * kHeadDim + r);
            const float4 v = __ldcg(o_at(k) + c * kRows + r);
            const float f = exp2_fast(mk - ref);
            ll = fmaf(f, __ldcg(at(k) + kRows * (kHeadDim + 1) + r), ll);
            if (mk != -INFINITY) {  // else nothing was written beside it
              o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
              o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
            }
          }
          const float inv = ll == 0.f ? 0.f : 1.f / ll;
          const size_t dst = (size_t)(w.c.qs + w.i0 + r / G) * a.hq + w.kvh * G + r % G;
          *reinterpret_cast<uint2*>(a.o + dst * kHeadDim + 4 * c) =
              make_uint2(pack_half2(__float2half_rn(o.x * inv), __float2half_rn(o.y * inv)),
                         pack_half2(__float2half_rn(o.z * inv), __float2half_rn(o.w * inv)));
          if (c == 0) a.lse[dst] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
        }
      }
      named_sync(1, 512);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Rows of 128 fp16 values in boxes of 64 columns (one 128-byte swizzle row).
bool encode(CUtensorMap* map, const uint16_t* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<uint16_t*>(base), dims,
                     strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G>
cudaError_t launch_g(const Args& a, cudaStream_t s) {
  CUtensorMap qm, km, vm;
  const cuuint64_t qd[3] = {kHeadDim, (cuuint64_t)a.hq, (cuuint64_t)a.total_q};
  const cuuint64_t qst[2] = {kHeadDim * 2, (cuuint64_t)a.hq * kHeadDim * 2};
  const cuuint32_t qbox[3] = {64, G, kTileRows / G};
  // Keys: a page is one copy of 8 rows x 64 columns, both halves of the columns, both groups of 8
  // rows, so that the groups of a key tile lie 2 KB apart whatever pages they come from (a copy per
  // page and half took 75 cycles each: 1200 a tile of K or V instead of 800).
  const cuuint64_t kd[4] = {64, 8, 2, (cuuint64_t)a.num_phys * a.hkv * (kPage / 8)};
  const cuuint64_t kst[3] = {kHeadDim * 2, 128, 8 * kHeadDim * 2};
  const cuuint32_t kbox[4] = {64, 8, 2, 2};
  if (!encode_fn() || !encode(&qm, a.q, 3, qd, qst, qbox) || !encode(&km, a.k, 4, kd, kst, kbox) ||
      !encode(&vm, a.v, 4, kd, kst, kbox))
    return cudaErrorNotSupported;
  cudaError_t e = cudaFuncSetAttribute(k_window_prefill<G>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  k_window_prefill<G><<<num_sms(), kThreads, kSmemBytes, s>>>(a, qm, km, vm);
  return cudaGetLastError();
}

}  // namespace

namespace {
uint32_t g_wait_limit = kWaitLimit;  // test knobs (twl_test_set_waits)
int g_stall = 0;
}  // namespace

void set_test_waits(uint32_t max_polls, int stall) {
  g_wait_limit = max_polls > 0 ? max_polls : kWaitLimit;
  g_stall = stall != 0;
}

size_t workspace_bytes() {
  return kCounterWords * sizeof(unsigned) + (size_t)num_sms() * 2 * kPartFloats * sizeof(float);
}

cudaError_t launch(Args a, void* ws, cudaStream_t s) {
  a.done = static_cast<unsigned*>(ws);  // a word per SM: fewer than kCounterWords
  a.part = reinterpret_cast<float*>(a.done + kCounterWords);
  a.wait_limit = g_wait_limit;
  a.stall = g_stall;
  switch (a.hq / a.hkv) {
    case 1: return launch_g<1>(a, s);
    case 2: return launch_g<2>(a, s);
    case 4: return launch_g<4>(a, s);
    case 8: return launch_g<8>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace prefill
}  // namespace twl
