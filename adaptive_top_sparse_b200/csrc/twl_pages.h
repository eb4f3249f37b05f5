// The page-table step and compaction of a paged cache (twl_pages.cu): arguments, launch.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "twl.h"

namespace twl {
namespace pages {

// Pages a pool may have: the CTAs keep a count per 256 pages in shared memory.
constexpr int kMaxPool = 1 << 23;
constexpr int kMaxBatch = 4096;

struct Pools {
  twl_page_pool pool[TWL_MAX_POOLS];
  int count;
};

struct Args {
  int* table;      // remap: read and written; compact: read
  int* table_out;  // compact (may equal table)
  int* seq_lens;
  const int* parent;
  const int* reserve;
  int* num_used;
  int batch, max_pages, num_phys;
  int sinks, window;
  unsigned wait_limit;  // polls before the barrier's wait gives up
  unsigned stall;       // test of that: the barrier waits for one CTA more than there are
  // workspace
  unsigned* sync;    // [4] arrivals, error bits, exits; zero between launches
  unsigned* bitmap;  // [words] used pages; zero between launches
  int* next;         // [batch][max_pages] the new table before its wanted pages
  int* slot;         // [4][batch] new length, pages needed, wanted pages, page to copy (or -1)
  uint32_t* flags;
};

size_t workspace_bytes(int batch, int max_pages);
void carve(Args& a, void* ws);
// Test knobs for the bounded wait (twl_test_set_waits).
void set_test_waits(uint32_t max_polls, int stall);
cudaError_t launch_remap(const Args& a, const Pools& p, cudaStream_t s);
cudaError_t launch_compact(const Args& a, const Pools& p, cudaStream_t s);

}  // namespace pages
}  // namespace twl
