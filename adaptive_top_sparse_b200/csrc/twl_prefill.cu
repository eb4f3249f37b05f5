// Attention of prompt chunks: the last q_len tokens of every sequence attend causally over a
// sliding window and the first (sink) tokens of the sequence's paged fp16 cache.
//
// Query row i of a chunk sits at position t = n - q_len + i and sees key j iff j <= t and
// (j < sinks or j > t - window).  o = softmax(scale q K^T) V over the seen keys in one pass: the
// running maximum and sum of each row rescale the accumulator when the maximum grows.
//
// Work split: the G heads of a kv-head share its keys, so the rows of a unit are (query, head)
// pairs, 64 per CTA; keys come in tiles of 64 tokens (4 pages).
#include "twl_common.cuh"
#include "twl_kernels.h"
#include "twl_prefill.h"

namespace twl {
namespace prefill {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kRows = 64, kKeys = 64, kThreads = 128;

__device__ __forceinline__ uint32_t sptr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Queries of sequence b's chunk, or 0 (and a flag) when its lengths cannot be served.
__device__ int chunk_len(const Args& a, int b, bool report) {
  const int s = a.q_start[b], e = a.q_start[b + 1], n = a.seq_lens[b];
  if (s < 0 || e < s || e > a.total_q || n < e - s || n > a.max_pages * kPage) {
    if (report) raise_flag(a.flags, TWL_FLAG_BAD_INDEX);
    return 0;
  }
  return e - s;
}

template <int G>
__global__ void __launch_bounds__(kThreads) k_window_prefill(const __grid_constant__ Args a) {
  constexpr int kQueries = kRows / G;
  __shared__ __align__(128) unsigned char ks[kKeys * 256], vs[kKeys * 256];
  __shared__ int scan_sh[33], s_b, s_unit, s_phys[kKeys / kPage];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, lg = lane >> 2, lt = lane & 3;

  // the unit: (sequence, 64 / G queries, kv-head)
  const int kvh = blockIdx.x % a.hkv, unit = blockIdx.x / a.hkv;
  if (tid == 0) s_b = -1;
  int carry = 0;
  for (int base = 0; base < a.batch; base += kThreads) {
    const int b = base + tid;
    const int c = b < a.batch ? (chunk_len(a, b, blockIdx.x == 0) + kQueries - 1) / kQueries : 0;
    int total;
    const int ex = carry + block_exclusive_scan(c, scan_sh, &total);
    if (unit >= ex && unit < ex + c) s_b = b, s_unit = unit - ex;
    carry += total;
  }
  __syncthreads();
  if (s_b < 0) return;
  const int b = s_b, i0 = s_unit * kQueries;
  const int qs = a.q_start[b], qn = a.q_start[b + 1] - qs, n = a.seq_lens[b];
  const int t0 = n - qn + i0, t1 = min(t0 + kQueries, n) - 1;  // positions of the unit's queries
  const int lo = t0 >= a.window ? t0 - a.window + 1 : 0;       // first key of any window

  uint32_t qa[8][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = warp * 16 + lg + 8 * r;
    const int i = i0 + row / G;
    const uint16_t* src = a.q + ((size_t)(qs + i) * a.hq + kvh * G + row % G) * kHeadDim + 2 * lt;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qa[kk][r] = i < qn ? *reinterpret_cast<const uint32_t*>(src + 16 * kk) : 0u;
      qa[kk][2 + r] = i < qn ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8) : 0u;
    }
  }
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;

  const int first = lo / kKeys, last = t1 / kKeys;
  const int sink_tiles = min((min(a.sinks, n) + kKeys - 1) / kKeys, first);
  for (int x = 0; x < sink_tiles + last - first + 1; ++x) {
    const int base = (x < sink_tiles ? x : first + x - sink_tiles) * kKeys;
    __syncthreads();
    if (tid < kKeys / kPage) {
      // a page is read when some query sees one of its keys
      const int p0 = base + tid * kPage;
      int ph = -1;
      if (p0 <= t1 && (p0 < a.sinks || p0 + kPage > lo))
        ph = load_phys(a.page_table, b, p0 / kPage, a.max_pages, a.num_phys, a.flags);
      s_phys[tid] = ph;
    }
    __syncthreads();
    for (int it = 0; it < kKeys * 16 / kThreads; ++it) {
      const int r = it * (kThreads / 16) + (tid >> 4), c = tid & 15, tok = base + r;
      const int ph = s_phys[r / kPage];
      const bool ok = ph >= 0 && tok <= t1 && (tok < a.sinks || tok >= lo);
      const size_t off = ok ? (((size_t)ph * a.hkv + kvh) * kPage + (r & 15)) * kHeadDim + c * 8 : 0;
      const int slot = r * 256 + ((c ^ (r & 7)) * 16);
      cp_async16(ks + slot, a.k + off, ok);
      cp_async16(vs + slot, a.v + off, ok);
    }
    cp_async_commit();
    cp_async_wait_all();
    __syncthreads();
    float s[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[j][c] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const int r = 8 * j + (lane >> 4) * 8 + (lane & 7);
        uint32_t f[4];
        ldmatrix4(f, sptr(ks) + r * 256 + (((2 * kk + ((lane >> 3) & 1)) ^ (r & 7)) * 16));
        mma_16816(s[j], qa[kk], f[0], f[1]);
        mma_16816(s[j + 1], qa[kk], f[2], f[3]);
      }
    }
    float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = base + 8 * j + 2 * lt + (c & 1);
        const int t = t0 + (warp * 16 + lg + 8 * (c >> 1)) / G;
        const bool see = key <= t && (key < a.sinks || key > t - a.window) && t < n &&
                         s_phys[(8 * j) / kPage] >= 0;
        s[j][c] = see ? s[j][c] * a.scale_log2 : -INFINITY;
        mt[c >> 1] = fmaxf(mt[c >> 1], s[j][c]);
      }
    float ref[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 1));
      mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 2));
      mt[r] = fmaxf(mt[r], m[r]);
      ref[r] = mt[r] == -INFINITY ? 0.f : mt[r];
      const float f = exp2f(m[r] - ref[r]);
      m[r] = mt[r];
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i][2 * r] *= f, o[i][2 * r + 1] *= f;
    }
    uint32_t p[4][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[j][c] = exp2f(s[j][c] - ref[c >> 1]);
        l[c >> 1] += s[j][c];
      }
      p[j >> 1][(j & 1) * 2] = pack_half2(__float2half_rn(s[j][0]), __float2half_rn(s[j][1]));
      p[j >> 1][(j & 1) * 2 + 1] = pack_half2(__float2half_rn(s[j][2]), __float2half_rn(s[j][3]));
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int r = 16 * kk + (lane & 15);
        uint32_t f[4];
        ldmatrix4_trans(f, sptr(vs) + r * 256 + (((i + (lane >> 4)) ^ (r & 7)) * 16));
        mma_16816(o[i], p[kk], f[0], f[1]);
        mma_16816(o[i + 1], p[kk], f[2], f[3]);
      }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = warp * 16 + lg + 8 * r, i = i0 + row / G;
    if (i >= qn) continue;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
    const size_t out = (size_t)(qs + i) * a.hq + kvh * G + row % G;
#pragma unroll
    for (int c = 0; c < 16; ++c)
      *reinterpret_cast<uint32_t*>(a.o + out * kHeadDim + 8 * c + 2 * lt) =
          pack_half2(__float2half_rn(o[c][2 * r] * inv), __float2half_rn(o[c][2 * r + 1] * inv));
    if (lt == 0) a.lse[out] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
  }
}

}  // namespace

size_t workspace_bytes(int batch, int hq, int hkv) { return 0; }

cudaError_t launch(const Args& a, void* ws, cudaStream_t s) {
  const int g = a.hq / a.hkv;
  const long long blocks =
      ((long long)a.total_q * g / kRows + a.batch) * a.hkv;  // at least the units of any split
#define TWL_PRE(G) k_window_prefill<G><<<(unsigned)blocks, kThreads, 0, s>>>(a)
  switch (g) {
    case 1: TWL_PRE(1); break;
    case 2: TWL_PRE(2); break;
    case 4: TWL_PRE(4); break;
    case 8: TWL_PRE(8); break;
    default: return cudaErrorInvalidValue;
  }
#undef TWL_PRE
  return cudaGetLastError();
}

}  // namespace prefill
}  // namespace twl
