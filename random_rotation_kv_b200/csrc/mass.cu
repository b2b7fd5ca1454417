// mass.cu — the attention weight that every cached token has drawn: softmax of each
// head's scores, summed over the query heads of a kv head and added to a running
// sum per token.
//
//     out[t] = decay·mass[t] + Σ_{h in group} e^{s[h,t] − m_h} / l_h,   l_h = Σ_t e^{s[h,t] − m_h}.
//
// One block per (sequence, kv head): a pass over the group's scores for the running
// maximum and sum of every head, a second one for the weights.  All fp32.
#include "evict.h"
#include "rrq_device.cuh"

namespace rrq {
namespace {

constexpr int kThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ int64_t clamp_len(const int32_t* lens, int64_t b, int64_t cap) {
  if (lens == nullptr) return cap;
  const int64_t n = lens[b];
  return n < 0 ? 0 : n > cap ? cap : n;
}

// (m, l) ⊕ (m2, l2), l in units of 2^m; −inf maxima carry l = 0.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float mx = fmaxf(m, m2);
  if (mx == -INFINITY) return;
  l = l * exp2f((m - mx) * kLog2e) + l2 * exp2f((m2 - mx) * kLog2e);
  m = mx;
}

__global__ void __launch_bounds__(kThreads) mass_kernel(const MassArgs a) {
  __shared__ float s_m[kThreads / 32], s_l[kThreads / 32];
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.x / a.hkv;
  const int64_t row = blockIdx.x;  // b·hkv + g
  const int64_t n = clamp_len(a.lens, b, a.T);
  const float* sc = a.scores + row * a.group * a.T;
  float* out = a.out + row * a.T;
  const float* in = a.mass ? a.mass + row * a.T : nullptr;
  for (int64_t t = tid; t < a.T; t += kThreads) {
    const float v = in ? in[t] : 0.f;
    out[t] = t < n ? a.decay * v : v;
  }
  for (int h = 0; h < a.group; ++h) {
    const float* s = sc + int64_t(h) * a.T;
    float m = -INFINITY, l = 0.f;
    for (int64_t t = tid; t < n; t += kThreads) m = fmaxf(m, s[t]);
    if (m != -INFINITY)
      for (int64_t t = tid; t < n; t += kThreads) l += exp2f((s[t] - m) * kLog2e);
    for (int o = 16; o > 0; o >>= 1)
      join(m, l, __shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, l, o));
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
    __syncthreads();
    m = -INFINITY;
    l = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) join(m, l, s_m[w], s_l[w]);
    if (m != -INFINITY) {
      const float inv = 1.f / l;
      for (int64_t t = tid; t < n; t += kThreads) out[t] += exp2f((s[t] - m) * kLog2e) * inv;
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t stream) {
  return launch_pdl(mass_kernel, dim3(unsigned(a.batch * a.hkv)), dim3(kThreads), 0, stream, a);
}

}  // namespace rrq
