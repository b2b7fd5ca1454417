// rope.h — arguments and launcher of the rotary-position kernel (rope.cu), called
// by the C ABI (api.cpp).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rrq {

constexpr int kRopeMaxPairs = 256;  // rot ≤ 512

struct RopeArgs {
  const void* x;             // [n × heads × d]
  void* y;                   // the same shape; may be x
  const int64_t* positions;  // [n]
  int64_t n;
  int heads, d, rot, interleaved;
  float cos_factor, sin_factor;  // factor, and ±factor (− for the transposed map)
};

// Frequency of pair i in units of 2^-64 turns per position.  A kernel parameter: launches
// with the 512 bytes of 64 pairs cost the host less than with 2 KB.
template <int N> struct RopeTurns {
  uint64_t turns[N];
};

cudaError_t launch_rope(const RopeArgs& a, const RopeTurns<kRopeMaxPairs>& f, int dtype, cudaStream_t stream);

}  // namespace rrq
