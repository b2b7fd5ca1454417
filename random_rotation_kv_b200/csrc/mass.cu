// mass.cu — the attention weight that every cached token has drawn: softmax of each
// head's scores, summed over the query heads of a kv head and added to a running
// sum per token.
//
//     out[t] = decay·mass[t] + Σ_{h in group} e^{s[h,t] − m_h} / l_h,   l_h = Σ_t e^{s[h,t] − m_h}.
//
// One cluster of up to 16 CTAs per (sequence, kv head), each with a run of tokens.  A CTA
// reads its scores once, into shared memory, and forms its own maximum and sum per
// head; the CTAs' pairs meet through distributed shared memory, and the weights then come
// from the scores that are still on the SM.  So every score crosses HBM once, which is
// what bounds the call (the group's heads cost 4 bytes a token each, the sums 8).
// Groups and lengths whose share does not fit shared memory read the scores again (from
// L2, as a rule).  All fp32; every sum's order is fixed by the sizes.
#include "cluster.cuh"
#include "evict.h"

namespace rrq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kMaxScores = 200 * 1024;  // bytes of scores a CTA keeps

__device__ __forceinline__ int64_t clamp_len(const int32_t* lens, int64_t b, int64_t cap) {
  if (lens == nullptr) return cap;
  const int64_t n = lens[b];
  return n < 0 ? 0 : n > cap ? cap : n;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  __syncthreads();  // red's previous readers are done
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = fmaxf(v, red[w]);
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v += red[w];
  return v;
}

// VEC: rows of scores and sums start on 16 bytes.  KEEP: the CTA's scores stay in shared
// memory (where they become e^{s − m}).  chunk: tokens per CTA, a multiple of 4.
template <bool VEC, bool KEEP>
__global__ void __launch_bounds__(kThreads) mass_kernel(const MassArgs a, int chunk, int size) {
  extern __shared__ __align__(16) float sm[];
  float* s_keep = sm;                                              // [group][chunk]
  float* s_ml = sm + (KEEP ? int64_t(a.group) * chunk : 0);        // [group][2]: maximum (times log2 e), sum
  float* s_f = s_ml + 2 * a.group;                                 // [group][2]: row maximum, factor
  __shared__ float red[kWarps];
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / size;  // b·hkv + g
  const int64_t b = row / a.hkv;
  const int64_t n = clamp_len(a.lens, b, a.T);
  const int64_t t0 = int64_t(blockIdx.x % size) * chunk;
  const int mine = int(t0 >= n ? 0 : n - t0 < chunk ? n - t0 : chunk);      // live tokens of this CTA
  const int all = int(t0 >= a.T ? 0 : a.T - t0 < chunk ? a.T - t0 : chunk);
  const float* sc = a.scores + row * a.group * a.T + t0;

  // ---- each head's maximum over the run, then its sum
  for (int h = 0; h < a.group; ++h) {
    const float* s = sc + int64_t(h) * a.T;
    float* k = s_keep + int64_t(h) * chunk;
    float m = -INFINITY;
    if constexpr (VEC) {
      const int full = mine & ~3;
#pragma unroll 4
      for (int t = tid * 4; t < full; t += kThreads * 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(s + t));
        if constexpr (KEEP) *reinterpret_cast<float4*>(k + t) = v;
        m = fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
      }
      if (full + tid < mine) {
        const float v = __ldg(s + full + tid);
        if constexpr (KEEP) k[full + tid] = v;
        m = fmaxf(m, v);
      }
    } else {
#pragma unroll 8
      for (int t = tid; t < mine; t += kThreads) {
        const float v = __ldg(s + t);
        if constexpr (KEEP) k[t] = v;
        m = fmaxf(m, v);
      }
    }
    m = block_max(m, red);
    float l = 0.f;
    if (m != -INFINITY) {
      for (int t = tid; t < mine; t += kThreads) {
        const float v = KEEP ? k[t] : __ldg(s + t);
        const float e = exp2_approx((v - m) * kLog2e);
        if constexpr (KEEP) k[t] = e;
        l += e;
      }
    } else if constexpr (KEEP) {
      for (int t = tid; t < mine; t += kThreads) k[t] = 0.f;
    }
    l = block_sum(l, red);
    if (tid == 0) {
      s_ml[2 * h] = m;
      s_ml[2 * h + 1] = l;
    }
  }
  // ---- the row's maximum and sum; factor = e^{m − row maximum} / row sum
  cluster_sync();
  for (int h = tid; h < a.group; h += kThreads) {
    const uint32_t at = smem_addr(s_ml + 2 * h);
    float m = -INFINITY, l = 0.f;
    for (int c = 0; c < size; ++c) m = fmaxf(m, __uint_as_float(ld_cluster(at, c)));
    if (m != -INFINITY)
      for (int c = 0; c < size; ++c)
        l += __uint_as_float(ld_cluster(at + 4, c)) * exp2_approx((__uint_as_float(ld_cluster(at, c)) - m) * kLog2e);
    s_f[2 * h] = m;
    s_f[2 * h + 1] = m == -INFINITY ? 0.f : (KEEP ? exp2_approx((s_ml[2 * h] - m) * kLog2e) : 1.f) / l;
  }
  cluster_sync();  // also: no CTA leaves while its pairs are read
  // ---- the sums
  const float* in = a.mass ? a.mass + row * a.T + t0 : nullptr;
  float* out = a.out + row * a.T + t0;
  if constexpr (VEC && KEEP) {
    const int full = mine & ~3;
    for (int t = tid * 4; t < full; t += kThreads * 4) {
      float4 v = in ? *reinterpret_cast<const float4*>(in + t) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int h = 0; h < a.group; ++h) {
        const float4 e = *reinterpret_cast<const float4*>(s_keep + int64_t(h) * chunk + t);
        const float f = s_f[2 * h + 1];
        w.x = fmaf(e.x, f, w.x), w.y = fmaf(e.y, f, w.y), w.z = fmaf(e.z, f, w.z), w.w = fmaf(e.w, f, w.w);
      }
      v.x = fmaf(a.decay, v.x, w.x), v.y = fmaf(a.decay, v.y, w.y), v.z = fmaf(a.decay, v.z, w.z), v.w = fmaf(a.decay, v.w, w.w);
      *reinterpret_cast<float4*>(out + t) = v;
    }
    if (full + tid < mine) {
      float w = 0.f;
      for (int h = 0; h < a.group; ++h) w = fmaf(s_keep[int64_t(h) * chunk + full + tid], s_f[2 * h + 1], w);
      out[full + tid] = fmaf(a.decay, in ? in[full + tid] : 0.f, w);
    }
  } else {
    for (int t = tid; t < mine; t += kThreads) {
      float w = 0.f;
      for (int h = 0; h < a.group; ++h) {
        if constexpr (KEEP) {
          w = fmaf(s_keep[int64_t(h) * chunk + t], s_f[2 * h + 1], w);
        } else {
          const float m = s_f[2 * h];
          if (m != -INFINITY) w = fmaf(exp2_approx((__ldg(sc + int64_t(h) * a.T + t) - m) * kLog2e), s_f[2 * h + 1], w);
        }
      }
      out[t] = fmaf(a.decay, in ? in[t] : 0.f, w);
    }
  }
  if (a.mass != a.out)  // behind the length: the sum as it was
    for (int t = mine + tid; t < all; t += kThreads) out[t] = in ? in[t] : 0.f;
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t stream) {
  const int64_t rows = a.batch * a.hkv;
  // a run per CTA short enough for its scores to stay in shared memory, where 16 CTAs can
  unsigned size = cluster_size(rows, a.T, 512);
  auto share = [&](unsigned c) { return ((a.T + c - 1) / c + 3) / 4 * 4; };
  while (size < 16 && size_t(share(size)) * a.group * 4 > kMaxScores) size *= 2;
  const int64_t chunk = share(size);
  const bool keep = size_t(chunk) * a.group * 4 <= kMaxScores;
  const bool vec = a.T % 4 == 0 && (reinterpret_cast<uintptr_t>(a.scores) | reinterpret_cast<uintptr_t>(a.mass) |
                                    reinterpret_cast<uintptr_t>(a.out)) % 16 == 0;
  const size_t smem = (keep ? size_t(chunk) * a.group : 0) * 4 + size_t(a.group) * 16;
  auto k = keep ? (vec ? mass_kernel<true, true> : mass_kernel<false, true>)
                : (vec ? mass_kernel<true, false> : mass_kernel<false, false>);
  return launch_cluster(k, dim3(unsigned(rows * size)), dim3(kThreads), size, smem, stream, a, int(chunk), int(size));
}

}  // namespace rrq
