// mass.cu — the attention weight that every cached token has drawn: softmax of each
// head's scores, summed over the query heads of a kv head and added to a running
// sum per token.
//
//     out[t] = decay·mass[t] + Σ_{h in group} e^{s[h,t] − m_h} / l_h,   l_h = Σ_t e^{s[h,t] − m_h}.
//
// One cluster of up to 16 CTAs per (sequence, kv head), each with a run of tokens.  A CTA
// reads its scores once, into shared memory (one bulk copy and barrier per head where rows
// start on 16 bytes, so a head is worked on while the next ones arrive).  Every thread
// keeps the maximum and sum of its own tokens and leaves e^{s − its maximum} in their
// place; the pairs meet within the CTA, then among the CTAs through distributed shared
// memory, and a thread's tokens take one factor per head.  So every score crosses HBM
// once, which is what bounds the call (the group's heads cost 4 bytes a token each, the
// sums 8).  Groups and lengths whose share does not fit shared memory read the scores
// again (from L2, as a rule).  All fp32; every sum's order is fixed by the sizes.
// 32 heads x 131072 scores in 8 groups: 11.1 us, 2.3 TB/s (80 of the 148 SMs, in clusters of 10);
// x 131073, whose rows start off 16 bytes (no bulk copies, 4-byte accesses): 24.9 us; 16 x 16
// heads x 2047: 7.2 us.
#include "cluster.cuh"
#include "evict.h"

namespace rrq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kMaxSmem = 224 * 1024;

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
// Maximum of the lanes' maxima and, over it, the sum of their sums l (of e^{s − own maximum});
// −inf maxima carry l = 0.
__device__ __forceinline__ void warp_join(float& m, float& l) {
  const float own = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  l = own == -INFINITY ? 0.f : l * exp2_approx((own - m) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
}

constexpr int kBars = 8;   // heads with a barrier of their own (the rest share the last one)
constexpr int kHold = 8;   // runs of four scores that a thread holds
constexpr int kHeads = 4;  // heads whose loads are in flight together (without bulk copies)

// VEC: rows of scores and sums start on 16 bytes.  KEEP: the CTA's scores stay in shared
// memory.  chunk: tokens per CTA, a multiple of 4.
template <bool VEC, bool KEEP>
__global__ void __launch_bounds__(kThreads) mass_kernel(const MassArgs a, int chunk, int size) {
  extern __shared__ __align__(16) float sm[];
  constexpr bool BULK = VEC && KEEP;
  float* s_keep = sm;                                              // [group][chunk]
  float* s_mt = sm + (KEEP ? int64_t(a.group) * chunk : 0);        // [group][threads]: a thread's maximum
  float* s_ml = s_mt + (KEEP ? a.group * kThreads : 0);            // [group][2]: maximum, sum
  float* s_f = s_ml + 2 * a.group;                                 // [group][2]: row maximum, 1 / row sum
  float* s_w = s_f + 2 * a.group;                                  // [group][warps][2]: maximum, sum
  __shared__ __align__(8) uint64_t s_bar[kBars];
  __shared__ int s_fail;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_fail = 0;
    for (int i = 0; i < kBars; ++i) mbarrier_init(smem_addr(&s_bar[i]), 1);
    fence_mbarrier_init();
  }
  pdl_release();
  pdl_wait();
  const int64_t row = blockIdx.x / size;  // b·hkv + g
  const int64_t b = row / a.hkv;
  const int64_t n = clamp_len(a.lens, b, a.T);
  const int64_t t0 = int64_t(blockIdx.x % size) * chunk;
  const int mine = int(t0 >= n ? 0 : n - t0 < chunk ? n - t0 : chunk);      // live tokens of this CTA
  const int all = int(t0 >= a.T ? 0 : a.T - t0 < chunk ? a.T - t0 : chunk);
  const float* sc = a.scores + row * a.group * a.T + t0;
  const float* in = a.mass ? a.mass + row * a.T + t0 : nullptr;
  float* out = a.out + row * a.T + t0;
  if constexpr (BULK) {
    // whole 16 bytes: a row's length is a multiple of 4 tokens, so nothing behind the row is read
    if (tid == 0 && mine > 0) {
      const uint32_t bytes = uint32_t((mine + 3) / 4 * 16);
      for (int h = 0; h < a.group; ++h) {
        const int bi = h < kBars ? h : kBars - 1;
        const uint32_t bar = smem_addr(&s_bar[bi]);
        if (h < kBars) mbarrier_expect_tx(bar, bytes * uint32_t(h == kBars - 1 ? a.group - h : 1));
        bulk_load(smem_addr(s_keep + int64_t(h) * chunk), sc + int64_t(h) * a.T, bytes, bar);
      }
      if (in) prefetch_l2(in, bytes);
    }
    __syncthreads();  // the barriers are there for the others
  }

  // ---- each head's maximum and sum over the run
  if constexpr (BULK) {
    for (int h = 0; h < a.group; ++h) {
      float* k = s_keep + int64_t(h) * chunk;
      float m = -INFINITY, l = 0.f;
      if (mine > 0 && h < kBars && !mbarrier_wait(smem_addr(&s_bar[h]), 0)) s_fail = 1;
      auto load = [&](int t) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (t < mine) v = *reinterpret_cast<const float4*>(k + t);
        if (t + 3 >= mine) {  // what the last copy brought from behind the length
          if (t + 1 >= mine) v.y = -INFINITY;
          if (t + 2 >= mine) v.z = -INFINITY;
          v.w = -INFINITY;
        }
        return v;
      };
      auto weigh = [&](float4 v, float c) {
        return make_float4(exp2_approx((v.x - c) * kLog2e), exp2_approx((v.y - c) * kLog2e), exp2_approx((v.z - c) * kLog2e),
                           exp2_approx((v.w - c) * kLog2e));
      };
      if (chunk <= kThreads * 4 * kHold) {  // a thread's scores fit its registers
        float4 v[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          v[i] = load((tid + i * kThreads) * 4);
          m = fmaxf(m, fmaxf(fmaxf(v[i].x, v[i].y), fmaxf(v[i].z, v[i].w)));
        }
        const float c = m == -INFINITY ? 0.f : m;  // every score −inf: e^{−inf} = 0
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int t = (tid + i * kThreads) * 4;
          if (t >= mine) break;
          v[i] = weigh(v[i], c);
          *reinterpret_cast<float4*>(k + t) = v[i];
          l += (v[i].x + v[i].y) + (v[i].z + v[i].w);
        }
      } else {
        for (int t = tid * 4; t < mine; t += kThreads * 4) {
          const float4 v = load(t);
          m = fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
        }
        const float c = m == -INFINITY ? 0.f : m;
        for (int t = tid * 4; t < mine; t += kThreads * 4) {
          const float4 v = weigh(load(t), c);
          *reinterpret_cast<float4*>(k + t) = v;
          l += (v.x + v.y) + (v.z + v.w);
        }
      }
      s_mt[h * kThreads + tid] = m;
      warp_join(m, l);
      if (lane == 0) s_w[2 * (h * kWarps + warp)] = m, s_w[2 * (h * kWarps + warp) + 1] = l;
    }
  } else {
    for (int h0 = 0; h0 < a.group; h0 += kHeads) {
      const float* s = sc + int64_t(h0) * a.T;
      float* k = s_keep + int64_t(h0) * chunk;
      const int hs = a.group - h0 < kHeads ? a.group - h0 : kHeads;
      float m[kHeads], l[kHeads];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll 4
      for (int t = tid; t < mine; t += kThreads) {
        float v[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) v[h] = h < hs ? __ldcg(s + int64_t(h) * a.T + t) : -INFINITY;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if constexpr (KEEP)
            if (h < hs) k[int64_t(h) * chunk + t] = v[h];
          m[h] = fmaxf(m[h], v[h]);
        }
      }
      for (int t = tid; t < mine; t += kThreads) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
          if (h < hs) {
            const float v = KEEP ? k[int64_t(h) * chunk + t] : __ldcg(s + int64_t(h) * a.T + t);
            const float e = m[h] != -INFINITY ? exp2_approx((v - m[h]) * kLog2e) : 0.f;
            if constexpr (KEEP) k[int64_t(h) * chunk + t] = e;
            l[h] += e;
          }
      }
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h < hs) {
          if constexpr (KEEP) s_mt[(h0 + h) * kThreads + tid] = m[h];
          warp_join(m[h], l[h]);
          if (lane == 0) s_w[2 * ((h0 + h) * kWarps + warp)] = m[h], s_w[2 * ((h0 + h) * kWarps + warp) + 1] = l[h];
        }
    }
  }
  __syncthreads();
  for (int h = warp; h < a.group; h += kWarps) {
    float m = lane < kWarps ? s_w[2 * (h * kWarps + lane)] : -INFINITY;
    float l = lane < kWarps ? s_w[2 * (h * kWarps + lane) + 1] : 0.f;
    warp_join(m, l);
    if (lane == 0) {
      s_ml[2 * h] = m;
      s_ml[2 * h + 1] = s_fail ? __uint_as_float(0x7fc00000u) : l;  // a copy that never came: NaN
    }
  }
  // ---- the row's maximum and sum (a warp per head, a lane per CTA)
  cluster_sync();
  for (int h = warp; h < a.group; h += kWarps) {
    const uint32_t at = smem_addr(s_ml + 2 * h);
    float m = lane < size ? __uint_as_float(ld_cluster(at, lane)) : -INFINITY;
    float l = lane < size ? __uint_as_float(ld_cluster(at + 4, lane)) : 0.f;
    warp_join(m, l);
    if (lane == 0) {
      s_f[2 * h] = m;
      s_f[2 * h + 1] = m == -INFINITY ? 0.f : 1.f / l;
    }
  }
  __syncthreads();
  cluster_arrive();  // this CTA has read the others' pairs
  // ---- the sums; a thread's factor of a head: e^{its maximum − row maximum} / row sum
  if constexpr (KEEP)
    for (int h = 0; h < a.group; ++h) {
      const float mt = s_mt[h * kThreads + tid];
      s_mt[h * kThreads + tid] = mt == -INFINITY ? 0.f : exp2_approx((mt - s_f[2 * h]) * kLog2e) * s_f[2 * h + 1];
    }
  if constexpr (BULK) {
#pragma unroll 4
    for (int t = tid * 4; t < mine; t += kThreads * 4) {
      const float4 v = in ? *reinterpret_cast<const float4*>(in + t) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int h = 0; h < a.group; ++h) {
        const float4 e = *reinterpret_cast<const float4*>(s_keep + int64_t(h) * chunk + t);
        const float f = s_mt[h * kThreads + tid];
        w.x = fmaf(e.x, f, w.x), w.y = fmaf(e.y, f, w.y), w.z = fmaf(e.z, f, w.z), w.w = fmaf(e.w, f, w.w);
      }
      w.x = fmaf(a.decay, v.x, w.x), w.y = fmaf(a.decay, v.y, w.y), w.z = fmaf(a.decay, v.z, w.z), w.w = fmaf(a.decay, v.w, w.w);
      if (t + 3 < mine) {
        *reinterpret_cast<float4*>(out + t) = w;
      } else {
        out[t] = w.x;
        if (t + 1 < mine) out[t + 1] = w.y;
        if (t + 2 < mine) out[t + 2] = w.z;
      }
    }
  } else {
    for (int t = tid; t < mine; t += kThreads) {
      float w = 0.f;
      for (int h = 0; h < a.group; ++h) {
        if constexpr (KEEP) {
          w = fmaf(s_keep[int64_t(h) * chunk + t], s_mt[h * kThreads + tid], w);
        } else {
          const float m = s_f[2 * h];
          if (m != -INFINITY) w = fmaf(exp2_approx((__ldcg(sc + int64_t(h) * a.T + t) - m) * kLog2e), s_f[2 * h + 1], w);
        }
      }
      out[t] = fmaf(a.decay, in ? in[t] : 0.f, w);
    }
  }
  if (a.mass != a.out)  // behind the length: the sum as it was
    for (int t = mine + tid; t < all; t += kThreads) out[t] = in ? in[t] : 0.f;
  cluster_wait();  // no CTA leaves while its pairs are read
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t stream) {
  const int64_t rows = a.batch * a.hkv;
  // 512 tokens per CTA at least (16 x 4 rows of 2047: 7.2 us, as with 128; with 2048 8.5)
  unsigned size = cluster_size(rows, a.T, 512);
  auto share = [&](unsigned c) { return ((a.T + c - 1) / c + 3) / 4 * 4; };
  const size_t pairs = size_t(a.group) * (16 + kWarps * 8);
  auto bytes = [&](unsigned c) { return (size_t(share(c)) + kThreads) * a.group * 4 + pairs; };  // with the scores kept
  // Runs whose scores take more than half of an SM's shared memory leave one CTA per SM.
  // Of clusters above 10 only 7 then run at a time (15 of 9, 11 of 10: the SMs of a GPC),
  // so 10 is tried before 16.
  while (size < 8 && bytes(size) > kMaxSmem) size *= 2;
  if (bytes(size) > kMaxSmem || (size == 16 && bytes(16) > 100 * 1024)) size = bytes(10) <= kMaxSmem ? 10 : 16;
  const int64_t chunk = share(size);
  const bool keep = bytes(size) <= kMaxSmem;
  const bool vec = a.T % 4 == 0 && (reinterpret_cast<uintptr_t>(a.scores) | reinterpret_cast<uintptr_t>(a.mass) |
                                    reinterpret_cast<uintptr_t>(a.out)) % 16 == 0;
  const size_t smem = keep ? bytes(size) : pairs;  // pairs: below 144 KB, as a group has at most kMassHeads heads
  static std::atomic<uint64_t> done[4];
  const int i = (keep ? 2 : 0) + (vec ? 1 : 0);
  auto k = keep ? (vec ? mass_kernel<true, true> : mass_kernel<false, true>)
                : (vec ? mass_kernel<true, false> : mass_kernel<false, false>);
  const cudaError_t e = allow_kernel(k, int(kMaxSmem), &done[i]);
  if (e != cudaSuccess) return e;
  return launch_cluster(k, dim3(unsigned(rows * size)), dim3(kThreads), size, smem, stream, a, int(chunk), int(size));
}

}  // namespace rrq
