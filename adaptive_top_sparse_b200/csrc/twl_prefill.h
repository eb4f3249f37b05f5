// Attention of chunks of many tokens over a window with sinks (twl_prefill.cu): arguments, launch.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twl {
namespace prefill {

struct Args {
  const uint16_t* q;   // [total_q][hq][128]
  const int* q_start;  // [batch + 1]
  int total_q, hq;
  const uint16_t *k, *v;
  const int* page_table;
  const int* seq_lens;
  int batch, hkv, max_pages, num_phys;
  int sinks, window;
  float scale_log2;  // score scale * log2(e)
  uint16_t* o;       // [total_q][hq][128]
  float* lse;        // [total_q][hq]
  uint32_t* flags;
  uint32_t wait_limit;  // polls before a wait gives up
  int stall;            // test of the waits: every second run's products never start
  // workspace, set by launch()
  unsigned* done;  // [SMs] arrived partials, by the run the unit starts in; zero between launches
  float* part;     // [SMs][2][256 rows x 130] partials of units cut by runs
};

size_t workspace_bytes();
// Test knobs for the bounded waits (twl_test_set_waits).
void set_test_waits(uint32_t max_polls, int stall);
cudaError_t launch(Args a, void* ws, cudaStream_t s);

}  // namespace prefill
}  // namespace twl
