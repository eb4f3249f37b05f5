// Attention of one query token per sequence over a sliding window and the first (sink) tokens of
// its paged cache: fp16 K/V, or K and V held in 4 bits.
//
// Query at position t = n - 1 sees key j iff j < n and (j < sinks or j >= n - window).  With
// s_j = scale q.k_j:  o = sum_j 2^(s_j' - m) v_j / sum_j 2^(s_j' - m),  s' = s log2(e).  A 4-bit
// row is x = c s + z (codes c, scale s, zero z of the row), so
//   q.k = s_k (q.c) + z_k sum(q)   and   sum_j p_j v_j = sum_j (p_j s_v,j) c_j + sum_j p_j z_v,j:
// only the integer codes go through the tensor cores, never a dequantised row.
//
// Bound: memory.  A token of one kv-head is 512 B (fp16) or 136 B (4-bit) and every byte is read
// once; the heads of a GQA group share the read.
//
// Work split: a page of 16 tokens (4-bit: two) of one (sequence, kv-head) group is a tile; the
// visible tiles of all groups form one flat list that is cut into runs, one per CTA, whatever the
// lengths.  A group that lies inside one run is finished there; a group cut by runs leaves one
// partial (max, sum, o) per CTA, and the CTA that arrives last merges them in CTA order (so the
// result does not depend on who is last).  Lengths stay on the device: each CTA derives the list
// from seq_lens.
//
// Inside a CTA the warps take the tiles in turn, each through its own ring of cp.async stages (no
// barrier in the loop), with transposed products so that the <= 8 heads of a group are the N = 8
// of mma.m16n8k16:  S^T = K Q^T (16 tokens x 8 heads), O^T = V^T P^T (16 dims x 8 heads); P^T
// comes from S^T by an 8x8 transpose in registers (movmatrix).
// Measured (one B200): 16 sequences of 8K-32K tokens, fp16, 205 us (6.15 TB/s, the copy rate is
// 6.55); 64 x 8K tokens of a 4-bit cache 183 us (3.1 TB/s).  There no unit is full (issue slots 52 %,
// ALU 50 %, DRAM 40 %, tensor 18 %): the bound is the latency of a warp's chain of scores, maximum,
// weights, transpose and V, 398 instructions a page, with 12 warps an SM (167 registers a thread; 12
// warps with two pages a step against 16 with one: 181, 185 us).
// Precision: o and lse are fp32 results, so P enters as hi + lo fp16 parts (22 bits).  With G <= 4
// the parts use the two halves of the N = 8 columns and cost nothing; G = 8 takes two products.
#include "twl_common.cuh"
#include "twl_kernels.h"
#include "twl_quant.cuh"
#include "twl_window.h"

namespace twl {
namespace window {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
// The running maximum of a head is only raised when a score exceeds it by more than this (log2
// units): weights stay below 2^8, far from fp16's largest value, and most tiles skip the rescale.
constexpr float kSlack = 8.f;
// Where a 4-bit code meets the tensor core as fp16 (see k_window_decode): two per word.
constexpr uint32_t kNibble = 0x00F000F0u;
// The maximum of a head that has seen nothing: finite, so that no difference with it is NaN, and
// below every finite score (2^92 at the largest scale, in magnitude).
constexpr float kNone = -1e30f;
// Runs that stay inside one group (see the kernel): tried for batches up to here, as a longer one
// cannot have a run for each sequence (148 SMs), and taken if the longest run is at most this many
// tiles longer than an equal share.  Measured on both sides, groups of 4 heads, 8 to 144 groups of 512
// to 32K tokens, equal and ragged, against runs of equal length:
//   tiles more   fp16 (16 tokens a tile)   4 bits (32)
//   up to 24     3-40 % faster             6-50 % faster
//   25 to 60     11 % faster to 3 % slower 28 % faster to 1 % slower
//   65 and more  5-80 % slower             3-60 % slower
constexpr int kAlignedBatch = 160;
constexpr int kJoinTiles = 24;
constexpr int kPartStride = 132;  // floats of one head's partial: o[128], max, sum, pad

template <bool INT4>
struct Cfg;
template <>
struct Cfg<false> {
  static constexpr int kWarps = 8, kStages = 3, kPages = 1, kTile = 8192, kRegs = 36;
};
template <>
struct Cfg<true> {
  static constexpr int kWarps = 12, kStages = 3, kPages = 2, kTile = 4352, kRegs = 38;
};

template <bool INT4>
constexpr size_t smem_bytes(int batch) {
  using C = Cfg<INT4>;
  return (size_t)C::kWarps * C::kStages * C::kTile + (size_t)(C::kWarps / 2) * C::kRegs * 128 +
         (size_t)(batch + 1) * 4;
}

// A (sequence, kv-head) group and its tiles [gs, ge) of the flat list.
struct Group {
  int b, kvh, gs, ge;
  int n, lo;     // keys; first key of the window
  int sink_pages, first_page;  // sink pages before the window's first page
  int pages;                   // of both kinds: kPages of them are a tile
};

__device__ __noinline__ Group group_of(const Args& a, const int* prefix, int f) {
  int x = 0, y = a.batch;  // prefix[x] * hkv <= f < prefix[y] * hkv
  while (y - x > 1) {
    const int mid = (x + y) >> 1;
    if ((long long)prefix[mid] * a.hkv <= f) x = mid;
    else y = mid;
  }
  Group g;
  g.b = x;
  const int per = prefix[x + 1] - prefix[x];
  g.kvh = (f - prefix[x] * a.hkv) / per;
  g.gs = prefix[x] * a.hkv + g.kvh * per;
  g.ge = g.gs + per;
  g.n = a.seq_lens[x] + a.appended;
  g.lo = max(0, g.n - a.window);
  g.first_page = g.lo / kPage;
  g.sink_pages = min((min(a.sinks, g.n) + kPage - 1) / kPage, g.first_page);
  g.pages = g.sink_pages + (g.n + kPage - 1) / kPage - g.first_page;
  return g;
}

// Visible pages of sequence b; 0 for an empty slot and for one that cannot be served (flagged
// by `report`).
__device__ int seq_pages(const Args& a, int b, bool report) {
  int n = a.seq_lens[b];
  if (a.appended) {
    const int j = n >> 4;
    int ph = -2;
    if (n >= 0 && j < a.max_pages) ph = a.page_table[(size_t)b * a.max_pages + j];
    if (n == 0 && ph == -1) return 0;  // an empty slot
    if (ph < 0 || ph >= a.num_phys) {
      if (report) raise_flag(a.flags, TWL_FLAG_BAD_INDEX);
      return 0;
    }
    ++n;
  }
  if (n < 0 || n > a.max_pages * kPage) {
    if (report) raise_flag(a.flags, TWL_FLAG_BAD_INDEX);
    return 0;
  }
  if (n == 0) return 0;
  const int first = max(0, n - a.window) / kPage;
  return min((min(a.sinks, n) + kPage - 1) / kPage, first) + (n + kPage - 1) / kPage - first;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// 16 bytes at src + OFF to shared memory at dst + OFF.
template <int OFF>
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;\n" ::"r"(dst), "l"(src),
               "n"(OFF));
}
// The same, or 16 zeros when `hide`.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool hide) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n"
      " cp.async.cg.shared.global [%0], [%1], 16, p;\n}\n" ::"r"(dst), "l"(src),
      "r"((uint32_t)hide));
}

// 16-byte slot of chunk c (0..3) of row r of a 4-bit V tile.  A lane reads 8 bytes of the rows of
// its four tokens (2t, 2t + 1, 2t + 8, 2t + 9); with this placement the 16 lanes of one shared
// memory phase touch every bank once.
__device__ __forceinline__ int v_slot(int r, int c) {
  return (r >> 1) * 8 + (((r ^ (r >> 2)) & 1) << 2) + (c ^ (r & 2));
}

// (c - 8) 2^-9 of two codes whose fp16 values are c 2^-9 / up.
__device__ __forceinline__ uint32_t centre(uint32_t codes, float up) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&codes), __float2half2_rn(up),
                            __float2half2_rn(-0x1p-6f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Softmax state and output accumulators of a warp.  Lane (g, t) = (lane / 4, lane % 4) holds the
// heads (N columns) 2t and 2t + 1; m is the same over g, l and z are this lane's tokens only.
struct State {
  float m[2], l[2], z[2], acc[8][4];
};

__device__ __forceinline__ void reset(State& st) {
#pragma unroll
  for (int c = 0; c < 2; ++c) st.m[c] = kNone, st.l[c] = 0.f, st.z[c] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) st.acc[i][c] = 0.f;
}

__device__ __forceinline__ void scale_state(State& st, float f0, float f1) {
  st.l[0] *= f0, st.l[1] *= f1, st.z[0] *= f0, st.z[1] *= f1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    st.acc[i][0] *= f0, st.acc[i][1] *= f1, st.acc[i][2] *= f0, st.acc[i][3] *= f1;
  }
}

// Raises the maxima to cover the tile's values t (t[0], t[1]: token g, heads 2t, 2t + 1; t[2],
// t[3]: token g + 8).
__device__ __forceinline__ void raise_max(State& st, const float (&t)[4]) {
  float f[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float x = fmaxf(t[c], t[c + 2]);
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
    const float m = fmaxf(st.m[c], x);
    f[c] = exp2_fast(st.m[c] - m);
    st.m[c] = m;
  }
  scale_state(st, f[0], f[1]);
}

__device__ __forceinline__ float max4(const float (&v)[4]) {
  return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
}

// P^T fragments (hi and lo parts) of the weights w (same order as t in raise_max).
template <int G>
__device__ __forceinline__ void p_fragments(const float (&w)[4], bool low, uint32_t (&hi)[2],
                                            uint32_t (&lo)[2]) {
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const __half2 h = __floats2half2_rn(w[2 * r], w[2 * r + 1]);
    const float2 f = __half22float2(h);
    const __half2 d = __floats2half2_rn(w[2 * r] - f.x, w[2 * r + 1] - f.y);
    const uint32_t hb = *reinterpret_cast<const uint32_t*>(&h);
    const uint32_t db = *reinterpret_cast<const uint32_t*>(&d);
    if constexpr (G == 8) {
      hi[r] = transpose8(hb);
      lo[r] = transpose8(db);
    } else {  // columns 0-3 carry the hi parts, 4-7 (lanes t >= 2) the lo parts of the same heads
      hi[r] = transpose8(low ? db : hb);
    }
  }
}

template <int G, bool INT4>
__global__ void __launch_bounds__(Cfg<INT4>::kWarps * 32, 1)
    k_window_decode(const __grid_constant__ Args a) {
  using C = Cfg<INT4>;
  constexpr int kWarps = C::kWarps, kStages = C::kStages, kTile = C::kTile, kBufs = kWarps / 2;
  constexpr int kPages = C::kPages;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem;
  float* buf = reinterpret_cast<float*>(smem + (size_t)kWarps * kStages * kTile);
  int* prefix = reinterpret_cast<int*>(buf + kBufs * C::kRegs * 32);
  __shared__ int scan_sh[33];
  __shared__ int tile_base[kWarps][kStages][kPages];  // first token of a stage's page; -1: none
  __shared__ int is_last;
  __shared__ int run_at[kAlignedBatch + 1];  // aligned runs before sequence b's

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lg = lane >> 2, lt = lane & 3;

  // ---- the flat list: prefix[b] = tiles per kv-head of the sequences before b
  int carry = 0;
  for (int base = 0; base < a.batch; base += blockDim.x) {
    const int b = base + tid;
    const int c = b < a.batch ? (seq_pages(a, b, blockIdx.x == 0) + kPages - 1) / kPages : 0;
    int total;
    const int ex = block_exclusive_scan(c, scan_sh, &total);
    if (b < a.batch) prefix[b] = carry + ex;
    carry += total;
  }
  if (tid == 0) prefix[a.batch] = carry;
  __syncthreads();
  const int total = prefix[a.batch] * a.hkv;

  // ---- sequences with no visible key
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    for (int i = tid; i < a.hq * kHeadDim; i += blockDim.x)
      a.o[(size_t)b * a.hq * kHeadDim + i] = 0.f;
    for (int i = tid; i < a.hq; i += blockDim.x) a.lse[(size_t)b * a.hq + i] = -INFINITY;
  }

  // A run has at least a tile for every warp (fewer partials to merge), unless the groups are
  // smaller than that.
  int runs = min(min((int)gridDim.x, total),
                 max((total + kWarps - 1) / kWarps, a.batch * a.hkv));
  // With few groups every run stays inside one: sequence b's groups get whole numbers of runs in
  // proportion to their tiles.  The longest run may then be longer than an equal share, but no CTA
  // joins twice; a second join costs about as much time as kJoinTiles tiles.
  bool aligned = false;
  if (a.batch <= kAlignedBatch && total > 0) {
    const int t = tid < a.batch ? prefix[tid + 1] - prefix[tid] : 0;
    const int c = t == 0 ? 0 : max(1, min(t * (int)gridDim.x / total, t / kWarps));
    int sum;
    const int ex = block_exclusive_scan(c * a.hkv, scan_sh, &sum);
    if (tid < a.batch) run_at[tid] = ex;
    if (tid == 0) run_at[a.batch] = sum;
    const int fair = (total + gridDim.x - 1) / gridDim.x;
    const int over = t != 0 && (t + c - 1) / c > max(fair, kWarps) + kJoinTiles;
    aligned = !__syncthreads_or(over) && sum <= (int)gridDim.x;
    if (aligned) runs = sum;
  }
  const int run = blockIdx.x;
  if (run < runs) {
    int f0, f1;
    int first_run = 0, last_run = 0;  // aligned: the runs of this one's group
    if (aligned) {
      int b = 0;
      while (run_at[b + 1] <= run) ++b;
      const int t = prefix[b + 1] - prefix[b], c = (run_at[b + 1] - run_at[b]) / a.hkv;
      const int kvh = (run - run_at[b]) / c, piece = (run - run_at[b]) % c;
      const int gs = prefix[b] * a.hkv + kvh * t;
      f0 = gs + t * piece / c;
      f1 = gs + t * (piece + 1) / c;
      first_run = run - piece;
      last_run = first_run + c - 1;
    } else {
      f0 = (int)((long long)total * run / runs);
      f1 = (int)((long long)total * (run + 1) / runs);
    }

    // ---- loads: the warp's next tile lf goes to the ring's stage ls; its page id is fetched one
    // tile ahead.  Addresses are running values: this is done for every 2 KB.
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring) + warp * kStages * kTile;
    const uint8_t *k_lane, *v_lane;  // the lane's 16 bytes of row 0 (fp16: of row lane / 16)
    const uint32_t* sz_lane = nullptr;
    uint32_t k_to, v_to;             // where they go in a stage
    if constexpr (INT4) {
      k_lane = a.kc + lane * 16;
      v_lane = a.vc + lane * 16;
      sz_lane = (lane < 4 ? a.ksz : a.vsz) + 4 * (lane & 3);
      k_to = lane * 16;
      v_to = 1024 + v_slot(lane >> 2, lane & 3) * 16;
    } else {
      k_lane = reinterpret_cast<const uint8_t*>(a.k) + lane * 16;
      v_lane = reinterpret_cast<const uint8_t*>(a.v) + lane * 16;
    }
    int lf = f0 + warp, ls = 0;
    int lgs, lend, lsink, lgap, lcount, lkvh, ln, llo;  // of the group of lf
    const int* ltable;
    auto enter = [&]() {
      const Group g = group_of(a, prefix, lf);
      lgs = g.gs;
      lend = g.ge;
      lsink = g.sink_pages;
      lgap = g.first_page - g.sink_pages;
      lcount = g.pages;
      lkvh = g.kvh;
      ln = g.n;
      llo = g.lo;
      ltable = a.page_table + (size_t)g.b * a.max_pages;
    };
    int lpage[kPages], lphys[kPages];  // -1 as a page: behind the group's last
    auto fetch = [&]() {
      if (lf >= f1) return;
      if (lf >= lend) enter();
#pragma unroll
      for (int h = 0; h < kPages; ++h) {
        const int i = (lf - lgs) * kPages + h;
        lpage[h] = i >= lcount ? -1 : i < lsink ? i : i + lgap;
        lphys[h] = i < lcount ? ltable[lpage[h]] : -1;
      }
    };
    if (lf < f1) enter(), fetch();
    auto issue = [&]() {
      if (lf < f1) {
#pragma unroll
        for (int h = 0; h < kPages; ++h) {
          const bool ok = (unsigned)lphys[h] < (unsigned)a.num_phys;
          if (lane == 0) {
            tile_base[warp][ls][h] = ok ? lpage[h] * kPage : -1;
            if (!ok && lpage[h] >= 0) raise_flag(a.flags, TWL_FLAG_BAD_INDEX);
          }
          const uint32_t st = ring_at + ls * kTile + h * (kTile / kPages);
          const uint32_t row0 = ok ? (uint32_t)(lphys[h] * a.hkv + lkvh) * kPage : 0u;
          if constexpr (INT4) {
            const uint8_t* ks = k_lane + (uint64_t)row0 * 64;
            const uint8_t* vs = v_lane + (uint64_t)row0 * 64;
            if (ok) {  // the codes of a page that is not there are not read
              copy16<0>(st + k_to, ks);
              copy16<512>(st + k_to, ks);
              copy16<0>(st + v_to, vs);
              copy16<512>(st + v_to, vs);  // rows r and r + 8 lie 512 bytes apart
              if (lane < 8) copy16<0>(st + 2048 + lane * 16, sz_lane + row0);
            }
          } else {
            const uint8_t* ks = k_lane + (uint64_t)row0 * 256;
            const uint8_t* vs = v_lane + (uint64_t)row0 * 256;
            const int c = lane & 15;
  #pragma unroll
            for (int it = 0; it < 8; ++it) {
              const int r = it * 2 + (lane >> 4), tok = lpage[h] * kPage + r;
              // rows nobody sees are zeroed: a weight of 0 times a stale infinity would be NaN
              const bool hide = !(ok && tok < ln && (tok < a.sinks || tok >= llo));
              const uint32_t to = st + r * 256 + ((c ^ (r & 7)) * 16);
              copy16_or_zero(to, ks + it * 512, hide);
              copy16_or_zero(to + 4096, vs + it * 512, hide);
            }
          }
        }
        lf += kWarps;
        fetch();
      }
      cp_async_commit();
      ls = ls + 1 == kStages ? 0 : ls + 1;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue();

    int f = f0 + warp, cs = 0;
    int gf = f0;  // start of the current segment
    while (gf < f1) {
      const Group g = group_of(a, prefix, gf);
      const int gend = min(g.ge, f1);
      // ---- the group's queries as the B operand: column = head (G <= 4: heads 0-3 twice)
      uint32_t qb[16];
      float qsum[2] = {0.f, 0.f};
      const float scale_k = a.scale_log2 * 0x1p20f;  // codes meet q as c 2^-20
      {
        const int h = G == 8 ? lg : (lg & 3);
        const uint16_t* qr = a.q + ((size_t)g.b * a.hq + g.kvh * G + h) * kHeadDim;
        const bool has = h < G;
        if constexpr (INT4) {
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (has) raw = *reinterpret_cast<const uint4*>(qr + 32 * lt + 8 * w);
            const uint32_t p[4] = {raw.x, raw.y, raw.z, raw.w};  // channel pairs (0,1) .. (6,7)
            qb[4 * w + 0] = __byte_perm(p[0], p[2], 0x5410);     // (0, 4)
            qb[4 * w + 1] = __byte_perm(p[1], p[3], 0x5410);     // (2, 6)
            qb[4 * w + 2] = __byte_perm(p[0], p[2], 0x7632);     // (1, 5)
            qb[4 * w + 3] = __byte_perm(p[1], p[3], 0x7632);     // (3, 7)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
              sum += x.x + x.y;
            }
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          // lane 4 h holds head h's sum; this lane needs columns 2t and 2t + 1
          qsum[0] = __shfl_sync(0xffffffffu, sum, 4 * (2 * lt)) * a.scale_log2;
          qsum[1] = __shfl_sync(0xffffffffu, sum, 4 * (2 * lt + 1)) * a.scale_log2;
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qb[2 * kk] = has ? *reinterpret_cast<const uint32_t*>(qr + 16 * kk + 2 * lt) : 0u;
            qb[2 * kk + 1] =
                has ? *reinterpret_cast<const uint32_t*>(qr + 16 * kk + 8 + 2 * lt) : 0u;
          }
        }
      }
      State st;
      reset(st);
      for (; f < gend; f += kWarps) {
        cp_async_wait<kStages - 2>();
        __syncwarp();  // every lane's copies have landed, and the stage read last is free
        issue();
        unsigned char* tile = ring + (warp * kStages + cs) * kTile;
        int base[kPages];
        bool clear = true, any = false;
#pragma unroll
        for (int h = 0; h < kPages; ++h) {
          base[h] = tile_base[warp][cs][h];
          any = any || base[h] >= 0;
          clear = clear && base[h] >= 0 && base[h] + kPage <= g.n &&
                  (base[h] >= g.lo || base[h] + kPage <= a.sinks);
        }
        cs = cs + 1 == kStages ? 0 : cs + 1;
        if (!any) continue;
        float x[kPages][4], w[kPages][4];
        auto sees = [&](int h, int r) {
          const int key = base[h] + lg + 8 * r;
          return base[h] >= 0 && key < g.n && (key < a.sinks || key >= g.lo);
        };
        if constexpr (INT4) {
          float sv[kPages][2], zv[kPages][2];
#pragma unroll
          for (int h = 0; h < kPages; ++h) {
            unsigned char* page = tile + h * 2176;
            uint32_t* ksz = reinterpret_cast<uint32_t*>(page + 2048);
            uint32_t* vsz = ksz + 16;
            if (a.appended && base[h] >= 0 && (unsigned)(g.n - 1 - base[h]) < (unsigned)kPage) {
              // the new token's row: quantised here, kept in the cache and patched into the tile
              const int r = (g.n - 1) & (kPage - 1);
              const int ph = a.page_table[(size_t)g.b * a.max_pages + base[h] / kPage];
              const size_t row = ((size_t)ph * a.hkv + g.kvh) * kPage + r;
              const size_t in = ((size_t)g.b * a.hkv + g.kvh) * kHeadDim + lane * 4;
              uint32_t sz;
              uint16_t code = quantize_row_warp(load_half4(a.k_new + in), &sz);
              reinterpret_cast<uint16_t*>(a.kc + row * 64)[lane] = code;
              reinterpret_cast<uint16_t*>(page + r * 64)[lane] = code;
              if (lane == 0) a.ksz[row] = sz, ksz[r] = sz;
              code = quantize_row_warp(load_half4(a.v_new + in), &sz);
              reinterpret_cast<uint16_t*>(a.vc + row * 64)[lane] = code;
              reinterpret_cast<uint16_t*>(page + 1024 + v_slot(r, lane >> 3) * 16)[lane & 7] = code;
              if (lane == 0) a.vsz[row] = sz, vsz[r] = sz;
              __syncwarp();
            }
            // A 4-bit code c at bits 4-7 of a half is the fp16 value c 2^-20 (fp16 is linear in its
            // bits up to 2^11).  Not at bits 0-3, where it is c 2^-24: the tensor core aligns
            // products by exponent, and ten leading zeros of a subnormal cost the sum ten bits
            // (measured: 6e-5 instead of 1e-6 of max|v|).
            float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
            const uint4 ra = *reinterpret_cast<const uint4*>(page + lg * 64 + lt * 16);
            const uint4 rb = *reinterpret_cast<const uint4*>(page + (lg + 8) * 64 + lt * 16);
            const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a0[4] = {wa[i] << 4 & kNibble, wb[i] << 4 & kNibble,
                                      wa[i] >> 4 & kNibble, wb[i] >> 4 & kNibble};
              const uint32_t a1[4] = {wa[i] & kNibble, wb[i] & kNibble, wa[i] >> 8 & kNibble,
                                      wb[i] >> 8 & kNibble};
              mma_16816(s0, a0, qb[4 * i], qb[4 * i + 1]);
              mma_16816(s1, a1, qb[4 * i + 2], qb[4 * i + 3]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(ksz + lg + 8 * r));
              const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(vsz + lg + 8 * r));
              sv[h][r] = vf.x, zv[h][r] = fmaf(8.f, vf.x, vf.y);  // V's codes enter as c - 8
              const float ks = kf.x * scale_k;
#pragma unroll
              for (int c = 0; c < 2; ++c)
                x[h][2 * r + c] = fmaf(ks, s0[2 * r + c] + s1[2 * r + c], kf.y * qsum[c]);
            }
          }
          if (!clear) {
#pragma unroll
            for (int h = 0; h < kPages; ++h)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (!sees(h, r)) {
                  x[h][2 * r] = x[h][2 * r + 1] = -INFINITY;
                  sv[h][r] = zv[h][r] = 0.f;
                }
          }
          // The weight that meets V's codes is w = p s_v, so the reference m covers the score and
          // s_v's exponent: w then stays below 2^9, and its two fp16 parts keep 22 bits whatever
          // the scale of V.  Checked on the outcome: it is raised for few tiles.
          float p[kPages][4];
          auto weigh = [&]() {
            bool high = false;
#pragma unroll
            for (int h = 0; h < kPages; ++h) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                p[h][i] = exp2_fast(x[h][i] - st.m[i & 1]);
                w[h][i] = p[h][i] * sv[h][i >> 1];
              }
              high = high || max4(w[h]) > 512.f || max4(p[h]) > 0x1p33f;
            }
            return high;
          };
          if (__any_sync(0xffffffffu, weigh())) {
#pragma unroll
            for (int h = 0; h < kPages; ++h) {
              float t[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                t[i] = x[h][i] +
                       (float)max((int)(__float_as_uint(sv[h][i >> 1]) >> 23) - 127, -24);
              raise_max(st, t);
            }
            weigh();
          }
#pragma unroll
          for (int h = 0; h < kPages; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              st.l[i & 1] += p[h][i];
              st.z[i & 1] = fmaf(p[h][i], zv[h][i >> 1], st.z[i & 1]);
            }
        } else {
          float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t kb = (uint32_t)__cvta_generic_to_shared(tile);
#pragma unroll
          for (int kk = 0; kk < 8; kk += 2) {
            const int r = lane & 15;
            uint32_t fa[4], fb[4];
            ldmatrix4(fa, kb + r * 256 + (((2 * kk + (lane >> 4)) ^ (r & 7)) * 16));
            ldmatrix4(fb, kb + r * 256 + (((2 * kk + 2 + (lane >> 4)) ^ (r & 7)) * 16));
            mma_16816(s0, fa, qb[2 * kk], qb[2 * kk + 1]);
            mma_16816(s1, fb, qb[2 * kk + 2], qb[2 * kk + 3]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) x[0][i] = (s0[i] + s1[i]) * a.scale_log2;
          if (!clear) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (!sees(0, r)) x[0][2 * r] = x[0][2 * r + 1] = -INFINITY;
          }
          // (as differences: those of large numbers are exact)
          if (__any_sync(0xffffffffu, fmaxf(x[0][0], x[0][2]) - st.m[0] > kSlack ||
                                          fmaxf(x[0][1], x[0][3]) - st.m[1] > kSlack))
            raise_max(st, x[0]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[0][i] = exp2_fast(x[0][i] - st.m[i & 1]);
            st.l[i & 1] += w[0][i];
          }
        }
#pragma unroll
        for (int h = 0; h < kPages; ++h) {
          uint32_t ph[2], pl[2];
          p_fragments<G>(w[h], lt >= 2, ph, pl);
          if constexpr (INT4) {
            const unsigned char* page = tile + h * 2176;
            const int c = lg >> 1;  // 16-byte chunk of the lane's 16 channels
            uint2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 2 * lt + (i & 1) + (i >> 1) * 8;
              v[i] = *reinterpret_cast<const uint2*>(page + 1024 + v_slot(r, c) * 16 +
                                                     (lg & 1) * 8);
            }
            const uint32_t x4[4] = {__byte_perm(v[0].x, v[1].x, 0x5410),
                                    __byte_perm(v[0].x, v[1].x, 0x7632),
                                    __byte_perm(v[0].y, v[1].y, 0x5410),
                                    __byte_perm(v[0].y, v[1].y, 0x7632)};
            const uint32_t y4[4] = {__byte_perm(v[2].x, v[3].x, 0x5410),
                                    __byte_perm(v[2].x, v[3].x, 0x7632),
                                    __byte_perm(v[2].y, v[3].y, 0x5410),
                                    __byte_perm(v[2].y, v[3].y, 0x7632)};
            // Block i: row g = channel 16 g + 2 i, row g + 8 = 16 g + 2 i + 1.  The codes enter as
            // (c - 8) 2^-9: without the offset the sum of codes and the sum of zeros are both far
            // larger than a diffuse head's o, and their difference is not an fp32 result any more
            // (measured at 8K tokens: 2e-5 of |o| off instead of 2e-6).
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t xx = i & 1 ? x4[i >> 1] >> 8 : x4[i >> 1];
              const uint32_t yy = i & 1 ? y4[i >> 1] >> 8 : y4[i >> 1];
              const uint32_t av[4] = {
                  centre(xx & 0x000F000Fu, 0x1p15f), centre(xx & kNibble, 0x1p11f),
                  centre(yy & 0x000F000Fu, 0x1p15f), centre(yy & kNibble, 0x1p11f)};
              mma_16816(st.acc[i], av, ph[0], ph[1]);
              if constexpr (G == 8) mma_16816(st.acc[i], av, pl[0], pl[1]);
            }
          } else {
            const uint32_t vb = (uint32_t)__cvta_generic_to_shared(tile) + 4096;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = (lane >> 4) * 8 + (lane & 7);
              uint32_t av[4];
              ldmatrix4_trans(av, vb + r * 256 + (((2 * i + ((lane >> 3) & 1)) ^ (r & 7)) * 16));
              // The tensor core truncates its sums: over the tiles of a long sequence that is a
              // bias (measured at 32K tokens: 2.3e-6 of |o| instead of 7e-7): it only sums a tile.
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16816(d, av, ph[0], ph[1]);
              if constexpr (G == 8) mma_16816(d, av, pl[0], pl[1]);
#pragma unroll
              for (int c = 0; c < 4; ++c) st.acc[i][c] += d[c];
            }
          }
        }
      }

      // ---- join the warps: the upper half into the lower half, then all threads over kBufs
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          st.l[c] += __shfl_xor_sync(0xffffffffu, st.l[c], o);
          if constexpr (INT4) st.z[c] += __shfl_xor_sync(0xffffffffu, st.z[c], o);
        }
      }
      float* mine = buf + (warp % kBufs) * C::kRegs * 32 + lane;
      auto put = [&]() {
#pragma unroll
        for (int i = 0; i < 32; ++i) mine[i * 32] = st.acc[i >> 2][i & 3];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mine[(32 + c) * 32] = st.m[c];
          mine[(34 + c) * 32] = st.l[c];
          if constexpr (INT4) mine[(36 + c) * 32] = st.z[c];
        }
      };
      if (warp >= kBufs) put();
      __syncthreads();
      if (warp < kBufs) {
        float fo[2], fm[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mo = mine[(32 + c) * 32], m = fmaxf(mo, st.m[c]);
          fo[c] = exp2_fast(mo - m);
          fm[c] = exp2_fast(st.m[c] - m);
          st.m[c] = m;
        }
        scale_state(st, fm[0], fm[1]);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          st.acc[i >> 2][i & 3] = fmaf(fo[i & 1], mine[i * 32], st.acc[i >> 2][i & 3]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          st.l[c] = fmaf(fo[c], mine[(34 + c) * 32], st.l[c]);
          if constexpr (INT4) st.z[c] = fmaf(fo[c], mine[(36 + c) * 32], st.z[c]);
        }
        put();
      }
      __syncthreads();
      const bool whole = g.gs >= f0 && g.ge <= f1;
      const int group = g.b * a.hkv + g.kvh;
      float* part = a.part + ((size_t)run * 2 + (g.gs < f0 ? 0 : 1)) * G * kPartStride;
      {
        // every warp joins 32 / kWarps of the accumulators, each lane its own columns
        constexpr int kMine = (32 + kWarps - 1) / kWarps;
        float m[2], l[2] = {0.f, 0.f}, z[2] = {0.f, 0.f}, o[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) o[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          m[c] = kNone;
#pragma unroll
          for (int k = 0; k < kBufs; ++k)
            m[c] = fmaxf(m[c], buf[(k * C::kRegs + 32 + c) * 32 + lane]);
        }
#pragma unroll
        for (int k = 0; k < kBufs; ++k) {
          const float* bk = buf + k * C::kRegs * 32 + lane;
          float s[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            s[c] = exp2_fast(bk[(32 + c) * 32] - m[c]);
            l[c] = fmaf(s[c], bk[(34 + c) * 32], l[c]);
            if constexpr (INT4) z[c] = fmaf(s[c], bk[(36 + c) * 32], z[c]);
          }
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const int reg = warp * kMine + i;
            if (reg < 32) o[i] = fmaf(reg & 1 ? s[1] : s[0], bk[reg * 32], o[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int reg = warp * kMine + i, c = reg & 1, h = 2 * lt + c;
          const float zc = c ? z[1] : z[0], lc = c ? l[1] : l[0];
          float v = o[i];
          if constexpr (G < 8) v += __shfl_xor_sync(0xffffffffu, v, 2);  // hi and lo parts
          int d;
          if constexpr (INT4) {
            d = 16 * lg + (reg >> 2) * 2 + (reg >> 1 & 1);
            v = fmaf(v, 0x1p9f, zc);
          } else {
            d = 16 * (reg >> 2) + 8 * (reg >> 1 & 1) + lg;
          }
          if (h < G && reg < 32) {
            const size_t row = (size_t)g.b * a.hq + g.kvh * G + h;
            if (whole) a.o[row * kHeadDim + d] = lc == 0.f ? 0.f : v / lc;
            else part[h * kPartStride + d] = v;
          }
        }
        if (warp == 0 && lg == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int h = 2 * lt + c;
            if (h >= G) continue;
            if (whole) {
              a.lse[(size_t)g.b * a.hq + g.kvh * G + h] =
                  l[c] == 0.f ? -INFINITY : (m[c] + log2f(l[c])) * kLn2;
            } else {
              part[h * kPartStride + kHeadDim] = m[c];
              part[h * kPartStride + kHeadDim + 1] = l[c];
            }
          }
        }
      }
      if (!whole) {
        // runs that hold tiles of the group: [first, last]
        const int first = aligned ? first_run : (int)(((long long)(g.gs + 1) * runs - 1) / total);
        const int last = aligned ? last_run : (int)(((long long)g.ge * runs - 1) / total);
        __threadfence();
        __syncthreads();
        if (tid == 0)
          is_last = atomicAdd(a.done + group, 1u) == (unsigned)(last - first);
        __syncthreads();
        if (is_last) {
          __threadfence();
          // Run `first` holds the group's start, so its partial is in its second slot; the others
          // began inside the group: first slot.  buf becomes the parts' weights and then the
          // columns of subsets of the parts, joined in a fixed order.
          const int parts = last - first + 1;
          auto at = [&](int c, int h) {
            return a.part + (((size_t)(first + c) * 2 + (c == 0 ? 1 : 0)) * G + h) * kPartStride;
          };
          float* wt = buf;                    // [parts][G] maxima, then weights
          float* ls = wt + parts * G;         // [parts][G] sums
          for (int e = tid; e < parts * G; e += kWarps * 32) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(at(e / G, e % G) + kHeadDim));
            wt[e] = ml.x;
            ls[e] = ml.y;
          }
          __syncthreads();
          constexpr int kSub = kWarps / G;    // warps per head
          const int h = warp % G, sub = warp / G;
          float m = kNone;
          for (int c = lane; c < parts; c += 32) m = fmaxf(m, wt[c * G + h]);
          m = warp_max(m);
          float l = 0.f;
          for (int c = lane; c < parts; c += 32)
            l = fmaf(exp2_fast(wt[c * G + h] - m), ls[c * G + h], l);
          l = warp_sum(l);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = sub; sub < kSub && c < parts; c += kSub) {
            const float s = exp2_fast(wt[c * G + h] - m);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(at(c, h) + 4 * lane));
            o.x = fmaf(s, v.x, o.x), o.y = fmaf(s, v.y, o.y);
            o.z = fmaf(s, v.z, o.z), o.w = fmaf(s, v.w, o.w);
          }
          float4* cols = reinterpret_cast<float4*>(buf + (2 * parts * G + 3) / 4 * 4);
          cols[warp * 32 + lane] = o;
          __syncthreads();
          if (sub == 0) {
#pragma unroll
            for (int k = 1; k < kSub; ++k) {
              const float4 v = cols[(k * G + h) * 32 + lane];
              o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
            }
            const size_t row = (size_t)g.b * a.hq + g.kvh * G + h;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            *reinterpret_cast<float4*>(a.o + row * kHeadDim + 4 * lane) =
                make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          }
          if (tid == 0) a.done[group] = 0u;
        }
      }
      __syncthreads();  // buf is free again
      gf = gend;
    }
    cp_async_wait_all();
  }

  if constexpr (INT4) {
    // ---- the last CTA to leave advances the lengths: by then every CTA has read them
    if (a.advance) {
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        is_last = atomicAdd(a.left, 1u) == gridDim.x - 1;
      }
      __syncthreads();
      if (is_last) {
        for (int b = tid; b < a.batch; b += blockDim.x)
          if (prefix[b + 1] != prefix[b]) a.seq_lens[b] += 1;
        if (tid == 0) *a.left = 0u;
      }
    }
  }
}

template <int G, bool INT4>
cudaError_t launch_g(const Args& a, cudaStream_t s) {
  // The attribute is the process's: every call sets the largest batch's, so that calls of other host
  // threads never find it below their own need.
  cudaError_t e = cudaFuncSetAttribute(k_window_decode<G, INT4>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem_bytes<INT4>(kWindowGroups));
  if (e != cudaSuccess) return e;
  k_window_decode<G, INT4>
      <<<num_sms(), Cfg<INT4>::kWarps * 32, smem_bytes<INT4>(a.batch), s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t workspace_bytes(int hq, int hkv) {
  const size_t g = hq / hkv;
  return kCounterWords * sizeof(unsigned) + (size_t)num_sms() * 2 * g * kPartStride * sizeof(float);
}

void carve(Args& a, void* ws) {
  a.done = static_cast<unsigned*>(ws);
  a.left = a.done + kWindowGroups;
  a.part = reinterpret_cast<float*>(a.done + kCounterWords);
}

cudaError_t launch(const Args& a, cudaStream_t s) {
  const bool int4 = a.kc != nullptr;
  switch (a.hq / a.hkv) {
    case 1: return int4 ? launch_g<1, true>(a, s) : launch_g<1, false>(a, s);
    case 2: return int4 ? launch_g<2, true>(a, s) : launch_g<2, false>(a, s);
    case 4: return int4 ? launch_g<4, true>(a, s) : launch_g<4, false>(a, s);
    case 8: return int4 ? launch_g<8, true>(a, s) : launch_g<8, false>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace window
}  // namespace twl
