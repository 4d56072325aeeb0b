// b8_attn.cuh -- what the attention kernels of the block-scaled 8-bit cache
// share.  Nothing here is part of the C ABI.
#pragma once

#include "b8_internal.cuh"

namespace kvq {

struct AttnArgs {
  kvq_b8_cache c;
  B8Queries q;
  B8Plan p;
  void *out;
  float *lse, *ws;  // ws: records [unit][split][row of the tile] of m, l, -, -, O[D]
  uint32_t *err;
  int polls;  // limit of the bounded waits
};

// rows of a CTA of the many-row kernel, and its workspace
int b8_prefill_rows(int head_dim);
size_t b8_prefill_workspace(int head_dim);
cudaError_t launch_b8_prefill(const AttnArgs &a, cudaStream_t s);

}  // namespace kvq
