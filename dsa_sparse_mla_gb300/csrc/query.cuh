// query.cuh — what the attention kernels share of scaling queries into fp16's range.
#pragma once

#include <stdint.h>

namespace hs {

// The exponent e by which a query's row is scaled (2^e) so that its latent values fit fp16, given the largest of its rotary
// values (|bf16| bits), which are scaled along. Where e would carry that value past 2^21, it is cut to what does not, though
// not below 0: the logits stay finite, and their scale back (2^-e) a normal number. Latent values that e then leaves
// below fp16's smallest step, 2^-25, are 2^-45 of the rotary ones: next to them they do not show in an fp32 sum.
__device__ __forceinline__ int query_exponent(int e, uint32_t rotary) {
  const int room = 20 - ((int)(rotary >> 7) - 127);
  return e <= 0 || e <= room ? e : (room > 0 ? room : 0);
}

}  // namespace hs
