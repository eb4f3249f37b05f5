// Attention of one token per sequence over a window with sinks (twl_window.cu): arguments, launch.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twl {
namespace window {

struct Args {
  const uint16_t* q;
  int hq;
  const uint16_t *k, *v;  // the fp16 cache (kc == nullptr) ...
  uint8_t *kc, *vc;       // ... or codes of the 4-bit cache
  uint32_t *ksz, *vsz;    // and its scale | zero << 16 of every row
  const uint16_t *k_new, *v_new;  // rows appended first (appended != 0)
  const int* page_table;
  int* seq_lens;  // written only with advance != 0
  int batch, hkv, max_pages, num_phys;
  int sinks, window;
  int appended, advance;
  float scale_log2;  // score scale * log2(e)
  float* o;
  float* lse;
  unsigned* done;  // [groups] arrived partials; zero between launches
  unsigned* left;  // CTAs that left (advance); zero between launches
  float* part;     // [SMs][2][G][132] partials of groups cut by runs
  uint32_t* flags;
};

size_t workspace_bytes(int hq, int hkv);
// Points the workspace arrays of `a` into `ws`, behind the header.
void carve(Args& a, void* ws);
cudaError_t launch(const Args& a, cudaStream_t s);

}  // namespace window
}  // namespace twl
