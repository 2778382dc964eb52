// qprefix.cuh — what the two kernels of decode over a shared prefix agree on.
#pragma once
#include <stdint.h>

namespace kascade {

// Tokens of sequence b that are attended to with the shared prefix: all P where it
// holds that many (lengths are cut to what the call and its block table hold), else
// none.
__device__ __forceinline__ int pfx_start(const int32_t* lens, int b, int P, int N, int max_blocks,
                                         int bs_shift) {
  const long long cap = min(static_cast<long long>(N), static_cast<long long>(max_blocks) << bs_shift);
  return min(static_cast<long long>(lens[b]), cap) >= P ? P : 0;
}

}  // namespace kascade
