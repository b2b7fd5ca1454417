// evict.h — arguments and launchers of the accumulated-weight and eviction kernels
// (mass.cu, evict.cu), called by the C ABI (api.cpp).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rrq {

constexpr int kMassHeads = 1024;  // query heads per kv head

struct MassArgs {
  const float* scores;  // [batch × hq × T]
  const int32_t* lens;  // [batch] or null
  const float* mass;    // [batch × hkv × T] or null; may be out
  float* out;           // [batch × hkv × T]
  int64_t batch, T;
  int hkv, group;
  float decay;
};
cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t stream);

struct EvictArgs {
  const float* mass;    // [batch × hkv × cap]
  const int32_t* lens;  // [batch] or null
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_norms;
  const float* v_norms;
  int32_t* index;       // [batch × hkv × keep]
  int32_t* out_lens;    // [batch]
  float* out_mass;      // [batch × hkv × keep] or null
  uint8_t* ok_codes;
  uint8_t* ov_codes;
  float* ok_norms;
  float* ov_norms;
  int64_t batch, cap, keep, sink, recent;
  int hkv, k_row, v_row;  // bytes of a K and a V code row
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace rrq
