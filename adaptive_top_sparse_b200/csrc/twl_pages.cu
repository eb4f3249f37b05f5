// Management of a paged cache: the page-table step (fork, free, grow, drop what left the window,
// copy the shared partial page) and the compaction of its pool.
//
// Both are one cooperative launch of one CTA per SM with one barrier over the grid.  Before it the
// CTAs read the old table and mark the pages that stay in use in a bitmap; behind it each CTA
// counts the bitmap (a bit per page: 8 KB for 64K pages), which gives every one of them the rank
// of any page and the page of any rank, so new pages and moves need no list, no sort and no
// further exchange, and come out in the same order whatever the CTAs' timing.  Nothing the caller
// owns is written before the barrier: a call that cannot be carried out changes nothing.
//
// Bound: the copies (read and write of every copied page).  A warp copies 4 KB at a time, 8 loads
// of 16 bytes per lane in flight; the pieces are dealt in equal contiguous runs over all warps.
#include "twl_common.cuh"
#include "twl_kernels.h"
#include "twl_pages.h"

namespace twl {
namespace pages {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 4096;           // bytes a warp copies at a time
constexpr int kGroupWords = 8;         // bitmap words per prefix entry (256 pages)
constexpr unsigned kSpinLimit = 1u << 24;  // polls (Args.wait_limit)
enum { kArrive = 0, kError = 1, kExit = 2, kSyncWords = 4 };
constexpr unsigned kNoPages = 1u << 30;

__host__ __device__ inline int groups_of(int num_phys) { return (num_phys + 255) / 256; }

// Barrier over the grid.  The launch is cooperative, so every CTA is resident; the limit only
// bounds a fault elsewhere.  Returns the error bits of all CTAs.
__device__ unsigned grid_barrier(const Args& a, unsigned mine, unsigned* sh) {
  __syncthreads();
  if (threadIdx.x == 0) {
    if (mine) atomicOr(a.sync + kError, mine);
    __threadfence();
    atomicAdd(a.sync + kArrive, 1u);
    unsigned seen = 0, polls = 0;
    const unsigned all = gridDim.x + a.stall;
    do {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(a.sync + kArrive));
    } while (seen < all && ++polls < a.wait_limit);
    __threadfence();
    unsigned e = __ldcg(a.sync + kError);
    if (seen < all) e |= TWL_FLAG_TIMEOUT;
    *sh = e;
  }
  __syncthreads();
  return *sh;
}

// The last CTA to leave clears the workspace for the next launch.
__device__ void leave(const Args& a, unsigned* sh) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    *sh = atomicAdd(a.sync + kExit, 1u);
  }
  __syncthreads();
  if (*sh != gridDim.x - 1) return;
  for (int i = threadIdx.x; i < groups_of(a.num_phys) * kGroupWords; i += kThreads)
    a.bitmap[i] = 0u;
  if (threadIdx.x < kSyncWords) a.sync[threadIdx.x] = 0u;
}

__device__ __forceinline__ void mark(const Args& a, int page) {
  atomicOr(a.bitmap + (page >> 5), 1u << (page & 31));
}

// prefix[i] = used pages before page 256 i, prefix[groups] = all of them.
__device__ void count_used(const Args& a, int* prefix, int* scan_sh) {
  const int groups = groups_of(a.num_phys);
  int carry = 0;
  for (int base = 0; base < groups; base += kThreads) {
    const int i = base + threadIdx.x;
    int c = 0;
    if (i < groups) {
      const uint4* w = reinterpret_cast<const uint4*>(a.bitmap) + 2 * (size_t)i;
      const uint4 x = __ldcg(w), y = __ldcg(w + 1);
      c = __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w) + __popc(y.x) + __popc(y.y) +
          __popc(y.z) + __popc(y.w);
    }
    int total;
    const int ex = block_exclusive_scan(c, scan_sh, &total);
    if (i < groups) prefix[i] = carry + ex;
    carry += total;
  }
  if (threadIdx.x == 0) prefix[groups] = carry;
  __syncthreads();
}

// Used pages below `page`.
__device__ int rank_used(const Args& a, const int* prefix, int page) {
  const int i = page >> 8;
  int c = prefix[i];
  for (int w = i * kGroupWords; w < (page >> 5); ++w) c += __popc(__ldcg(a.bitmap + w));
  if (page & 31) c += __popc(__ldcg(a.bitmap + (page >> 5)) & ((1u << (page & 31)) - 1u));
  return c;
}

// The page of rank r among the used (or free) pages; r must be below their number.
template <bool USED>
__device__ int page_of_rank(const Args& a, const int* prefix, int r) {
  int x = 0, y = groups_of(a.num_phys);  // before(x) <= r < before(y)
  while (y - x > 1) {
    const int mid = (x + y) >> 1;
    const int before = USED ? prefix[mid] : 256 * mid - prefix[mid];
    if (before <= r) x = mid;
    else y = mid;
  }
  r -= USED ? prefix[x] : 256 * x - prefix[x];
  const uint4* p = reinterpret_cast<const uint4*>(a.bitmap) + 2 * (size_t)x;
  const uint4 u = __ldcg(p), v = __ldcg(p + 1);
  const unsigned w[kGroupWords] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  int page = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < kGroupWords; ++i) {
    unsigned bits = USED ? w[i] : ~w[i];
    const int c = __popc(bits);
    if (!found && r < c) {
      found = true;
      for (int k = 0; k < r; ++k) bits &= bits - 1u;
      page = (x * kGroupWords + i) * 32 + __ffs(bits) - 1;
    }
    if (!found) r -= c;
  }
  return page;
}

__device__ __forceinline__ void copy_piece(const char* src, char* dst, int bytes, int lane) {
  const int n = bytes >> 4;  // 16-byte units, at most 256
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  uint4 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i * 32 + lane < n) x[i] = __ldcs(s + i * 32 + lane);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i * 32 + lane < n) d[i * 32 + lane] = x[i];
}

// Copies `count` pages of every pool: ends(k, &from, &to) names the k-th copy.  Pieces are
// numbered (k, pool, piece) and each warp takes one contiguous run of them.
template <typename Ends>
__device__ void copy_pages(const Pools& p, int count, Ends ends) {
  const int lane = threadIdx.x & 31;
  long long per = 0;
  for (int i = 0; i < p.count; ++i) per += (p.pool[i].page_bytes + kPiece - 1) / kPiece;
  const long long warps = (long long)gridDim.x * kWarps;
  const long long w = (long long)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  const long long total = per * count;
  long long at = total * w / warps;
  const long long end = total * (w + 1) / warps;
  if (at >= end) return;
  int k = (int)(at / per), pool = 0;
  long long piece = at % per;
  while (piece >= (p.pool[pool].page_bytes + kPiece - 1) / kPiece)
    piece -= (p.pool[pool++].page_bytes + kPiece - 1) / kPiece;
  int from, to;
  ends(k, &from, &to);
  for (; at < end; ++at) {
    const long long bytes = p.pool[pool].page_bytes, off = piece * kPiece;
    char* base = static_cast<char*>(p.pool[pool].data);
    copy_piece(base + from * bytes + off, base + to * bytes + off,
               (int)(bytes - off < kPiece ? bytes - off : kPiece), lane);
    if (off + kPiece >= bytes) {
      piece = 0;
      if (++pool == p.count) {
        pool = 0;
        ++k;
        if (at + 1 < end) ends(k, &from, &to);
      }
    } else {
      ++piece;
    }
  }
}

// ------------------------------------------------------------------ the page-table step
// What slot b becomes.
struct Slot {
  int src;      // its parent, or -1: freed
  int n;        // its length
  int need;     // pages of its length and reserve
  bool keeper;  // it keeps the parent's partial page (the parent's own slot, else its lowest fork)
  bool own;     // it is its own parent
};

__device__ Slot slot_of(const Args& a, const int* keeper, int b, unsigned* err) {
  Slot s;
  s.src = a.parent[b];
  s.n = 0;
  const int reserve = a.reserve ? a.reserve[b] : 0;
  if (s.src < -1 || s.src >= a.batch || reserve < 0) {
    *err |= TWL_FLAG_BAD_INDEX;
    s.src = -1;
  }
  if (s.src >= 0) {
    s.n = a.seq_lens[s.src];
    if (s.n < 0 || s.n > a.max_pages * kPage) {
      *err |= TWL_FLAG_BAD_INDEX;
      s.n = 0;
    }
  }
  const long long need = ((long long)s.n + max(reserve, 0) + kPage - 1) / kPage;
  if (need > a.max_pages) *err |= TWL_FLAG_BAD_INDEX;
  s.need = (int)min(need, (long long)a.max_pages);
  s.own = s.src == b;
  s.keeper = s.src >= 0 && keeper[s.src] == b;
  return s;
}

// Entry j of slot s before its wanted pages: a page it goes on holding, else -1.  *from: the page
// whose rows the slot has to copy into a new one, if this entry is its shared partial page.
__device__ __forceinline__ int next_entry(const Args& a, const Slot& s, int j, int* from,
                                          unsigned* err) {
  if (s.src < 0 || j >= s.need) return -1;
  const int whole = s.n / kPage, held = (s.n + kPage - 1) / kPage;
  if (j >= held && !s.own) return -1;
  if (j < whole) {
    // a page none of whose tokens a later query sees is dropped (the next query is at position n)
    const int first = j * kPage, last = first + kPage - 1;
    if (first >= a.sinks && last <= s.n - a.window) return -1;
  }
  const int page = a.table[(size_t)s.src * a.max_pages + j];
  if (page >= a.num_phys) {
    *err |= TWL_FLAG_BAD_INDEX;
    return -1;
  }
  if (page < 0) return -1;
  if (j == whole && j < held && !s.keeper) {
    *from = page;
    return -1;
  }
  return page;
}

__global__ void __launch_bounds__(kThreads, 1)
    k_remap(const __grid_constant__ Args a, const __grid_constant__ Pools pools) {
  extern __shared__ int sh[];
  __shared__ int scan_sh[33];
  __shared__ unsigned sh_word;
  const int groups = groups_of(a.num_phys);
  int* keeper = sh;              // [batch]; behind the barrier: prefix of the wanted pages
  int* copies = sh + a.batch + 1;  // [batch] slots that copy
  int* prefix = copies + a.batch;  // [groups + 1]
  int* n_of = a.slot;
  int* need_of = n_of + a.batch;
  int* wants_of = need_of + a.batch;
  int* from_of = wants_of + a.batch;
  const int tid = threadIdx.x, lane = tid & 31;
  unsigned err = 0;

  for (int b = tid; b < a.batch; b += kThreads) keeper[b] = 0x7FFFFFFF;
  __syncthreads();
  for (int b = tid; b < a.batch; b += kThreads) {
    const int p = a.parent[b];
    if (p >= 0 && p < a.batch && a.parent[p] != p) atomicMin(keeper + p, b);
    if (p == b) keeper[b] = b;  // no atomicMin reaches this entry
  }
  __syncthreads();

  // ---- what stays: the entries of 512 logical pages of a slot at a time.  What a thread found in
  // its first stretch, and a warp for its first slot, stays in registers over the barrier (that is
  // all of it unless the tables are large).
  const int chunks = (a.max_pages + kThreads - 1) / kThreads;
  int my_page = -1;
  Slot my_slot = {-1, 0, 0, false, false};
  for (int item = blockIdx.x; item < a.batch * chunks; item += gridDim.x) {
    const int b = item / chunks, j = (item % chunks) * kThreads + tid;
    const Slot s = slot_of(a, keeper, b, &err);
    int page = -1;
    if (j < a.max_pages) {
      int from;
      page = next_entry(a, s, j, &from, &err);
      a.next[(size_t)b * a.max_pages + j] = page;
      if (page >= 0) mark(a, page);
    }
    if (item == (int)blockIdx.x) my_page = page, my_slot = s;
  }
  // ---- what is wanted: a warp per slot, over the pages behind its whole ones
  const int warps = gridDim.x * kWarps, warp = blockIdx.x + gridDim.x * (tid >> 5);
  int my_n = 0, my_need = 0;
  unsigned my_want = 0;  // of its first 32 such pages
  for (int b = warp; b < a.batch; b += warps) {
    const Slot s = slot_of(a, keeper, b, &err);
    int wants = 0, copy = -1;
    for (int j = s.n / kPage + lane; j < s.need; j += 32) {
      int from = -1;
      if (next_entry(a, s, j, &from, &err) < 0) {
        ++wants;
        if (b == warp && j < s.n / kPage + 32) my_want = 1;
      }
      if (from >= 0) copy = from;
    }
    wants = __reduce_add_sync(0xffffffffu, wants);
    copy = __reduce_max_sync(0xffffffffu, copy);
    if (b == warp) my_n = s.n, my_need = s.need;
    if (lane == 0) {
      n_of[b] = s.n;
      need_of[b] = s.need;
      wants_of[b] = wants;
      from_of[b] = copy;
    }
  }
  my_want = __ballot_sync(0xffffffffu, my_want != 0);
  err = __syncthreads_or(err) ? TWL_FLAG_BAD_INDEX : 0u;
  err = grid_barrier(a, err, &sh_word);

  if (err == 0) {
    // the slots' counts are under way while the bitmap is counted
    int my_wants = tid < a.batch ? __ldcg(wants_of + tid) : 0;
    int my_from = tid < a.batch ? __ldcg(from_of + tid) : -1;
    count_used(a, prefix, scan_sh);
    int* want_prefix = keeper;
    int wanted = 0, ncopies = 0;
    for (int base = 0; base < a.batch; base += kThreads) {
      const int b = base + tid;
      if (base > 0) {
        my_wants = b < a.batch ? __ldcg(wants_of + b) : 0;
        my_from = b < a.batch ? __ldcg(from_of + b) : -1;
      }
      const int c = my_wants, f = my_from >= 0 ? 1 : 0;
      int total;
      int ex = block_exclusive_scan(c, scan_sh, &total);
      if (b < a.batch) want_prefix[b] = wanted + ex;
      wanted += total;
      ex = block_exclusive_scan(f, scan_sh, &total);
      if (f) copies[ncopies + ex] = b;
      ncopies += total;
    }
    __syncthreads();
    if (wanted > a.num_phys - prefix[groups]) {
      err = kNoPages;
    } else {
      // ---- the new table: entry by entry, then the wanted pages in (slot, logical page) order
      for (int item = blockIdx.x; item < a.batch * chunks; item += gridDim.x) {
        const int b = item / chunks, j = (item % chunks) * kThreads + tid;
        if (j < a.max_pages) {
          const size_t i = (size_t)b * a.max_pages + j;
          const bool mine = item == (int)blockIdx.x;
          const int page = mine ? my_page : __ldcg(a.next + i);
          const int n = mine ? my_slot.n : __ldcg(n_of + b);
          const int need = mine ? my_slot.need : __ldcg(need_of + b);
          if (page >= 0 || j < n / kPage || j >= need) a.table[i] = page;
        }
      }
      for (int b = warp; b < a.batch; b += warps) {
        int rank = want_prefix[b];
        const bool mine = b == warp;
        const int n = mine ? my_n : __ldcg(n_of + b), need = mine ? my_need : __ldcg(need_of + b);
        for (int base = n / kPage; base < need; base += 32) {
          const int j = base + lane;
          const size_t i = (size_t)b * a.max_pages + j;
          const unsigned all =
              mine && base == n / kPage
                  ? my_want
                  : __ballot_sync(0xffffffffu, j < need && __ldcg(a.next + i) < 0);
          if (all >> lane & 1u)
            a.table[i] = page_of_rank<false>(a, prefix, rank + __popc(all & ((1u << lane) - 1u)));
          rank += __popc(all);
        }
        if (lane == 0) a.seq_lens[b] = n;
      }
      // ---- the partial pages: a copying slot's first wanted page is its copy
      copy_pages(pools, ncopies, [&](int k, int* from, int* to) {
        *from = __ldcg(from_of + copies[k]);
        *to = page_of_rank<false>(a, prefix, want_prefix[copies[k]]);
      });
    }
  }
  if (err != 0 && blockIdx.x == 0 && tid == 0)
    raise_flag(a.flags, err == kNoPages ? TWL_FLAG_NO_PAGES : err);
  leave(a, &sh_word);
}

// ------------------------------------------------------------------ compaction
__global__ void __launch_bounds__(kThreads, 1)
    k_compact(const __grid_constant__ Args a, const __grid_constant__ Pools pools) {
  extern __shared__ int prefix[];  // [groups + 1]
  __shared__ int scan_sh[33];
  __shared__ unsigned sh_word;
  const int tid = threadIdx.x;
  const long long entries = (long long)a.batch * a.max_pages;
  unsigned err = 0;
  for (long long i = (long long)blockIdx.x * kThreads + tid; i < entries;
       i += (long long)gridDim.x * kThreads) {
    const int page = a.table[i];
    if (page >= a.num_phys) err = TWL_FLAG_BAD_INDEX;
    else if (page >= 0) mark(a, page);
  }
  err = __syncthreads_or(err) ? TWL_FLAG_BAD_INDEX : 0u;
  err = grid_barrier(a, err, &sh_word);
  if (err == 0) {
    count_used(a, prefix, scan_sh);
    // the used pages at or behind `used` move, in order, into the free ones before it
    const int used = prefix[groups_of(a.num_phys)];
    const int stay = used < a.num_phys ? rank_used(a, prefix, used) : used;
    if (blockIdx.x == 0 && tid == 0) *a.num_used = used;
    for (long long i = (long long)blockIdx.x * kThreads + tid; i < entries;
         i += (long long)gridDim.x * kThreads) {
      int page = a.table[i];
      if (page >= used) page = page_of_rank<false>(a, prefix, rank_used(a, prefix, page) - stay);
      a.table_out[i] = page;
    }
    copy_pages(pools, used - stay, [&](int k, int* from, int* to) {
      *from = page_of_rank<true>(a, prefix, stay + k);
      *to = page_of_rank<false>(a, prefix, k);
    });
  } else if (blockIdx.x == 0 && tid == 0) {
    raise_flag(a.flags, err);
  }
  leave(a, &sh_word);
}

size_t remap_smem(int batch, int num_phys) {
  return (2 * (size_t)batch + 1 + groups_of(num_phys) + 1) * sizeof(int);
}
size_t compact_smem(int num_phys) { return ((size_t)groups_of(num_phys) + 1) * sizeof(int); }

unsigned g_wait_limit = kSpinLimit;  // test knobs (twl_test_set_waits)
unsigned g_stall = 0;

// most: the kernel's need for the largest batch and pool.  The attribute is the process's, so every
// call sets the same value: calls of other host threads never find it below their own need.
cudaError_t launch(const void* kernel, Args a, const Pools& p, size_t smem, size_t most,
                   cudaStream_t s) {
  a.wait_limit = g_wait_limit;
  a.stall = g_stall;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  void* args[] = {&a, const_cast<Pools*>(&p)};
  return cudaLaunchCooperativeKernel(kernel, dim3(num_sms()), dim3(kThreads), args, smem, s);
}

}  // namespace

void set_test_waits(uint32_t max_polls, int stall) {
  g_wait_limit = max_polls > 0 ? max_polls : kSpinLimit;
  g_stall = stall != 0;
}

// The bitmap has room for the largest pool: what is zero between launches lies in one place whatever
// the call's sizes, so that one workspace serves them all.
size_t workspace_bytes(int batch, int max_pages) {
  return kSyncWords * 4 + kMaxPool / 8 + (size_t)batch * max_pages * 4 + (size_t)batch * 16;
}

void carve(Args& a, void* ws) {
  a.sync = static_cast<unsigned*>(ws);
  a.bitmap = a.sync + kSyncWords;  // 16-byte aligned: read as uint4
  a.next = reinterpret_cast<int*>(a.bitmap + kMaxPool / 32);
  a.slot = a.next + (size_t)a.batch * a.max_pages;
}

cudaError_t launch_remap(const Args& a, const Pools& p, cudaStream_t s) {
  return launch(reinterpret_cast<const void*>(k_remap), a, p, remap_smem(a.batch, a.num_phys),
                remap_smem(kMaxBatch, kMaxPool), s);
}

cudaError_t launch_compact(const Args& a, const Pools& p, cudaStream_t s) {
  return launch(reinterpret_cast<const void*>(k_compact), a, p, compact_smem(a.num_phys),
                compact_smem(kMaxPool), s);
}

}  // namespace pages
}  // namespace twl
