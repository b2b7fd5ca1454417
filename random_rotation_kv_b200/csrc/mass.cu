// mass.cu — the attention weight that every cached token has drawn: softmax of each
// head's scores, summed over the query heads of a kv head and added to a running
// sum per token.
//
//     out[t] = decay·mass[t] + Σ_{h in group} e^{s[h,t] − m_h} / l_h,   l_h = Σ_t e^{s[h,t] − m_h}.
//
// One cluster of up to 16 CTAs per (sequence, kv head), each with a run of tokens.  A CTA
// reads its scores once, into shared memory (one bulk copy per head where rows start on 16
// bytes), and forms its own maximum and sum per head; the CTAs' pairs meet through
// distributed shared memory, and the weights then come from the scores that are still on
// the SM.  So every score crosses HBM once, which is what bounds the call (the group's
// heads cost 4 bytes a token each, the sums 8).  Groups and lengths whose share does not
// fit shared memory read the scores again (from L2, as a rule).  All fp32; every sum's order
// is fixed by the sizes.
#include "cluster.cuh"
#include "evict.h"

namespace rrq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kMaxScores = 216 * 1024;  // bytes of scores a CTA keeps
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
// Maximum (or sum) of each of H values over the block, in red[H][warps]; all threads get it.
template <int H, bool MAX> __device__ __forceinline__ void block_reduce(float (&v)[H], float (*red)[kWarps]) {
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(kFull, v[h], o);
      v[h] = MAX ? fmaxf(v[h], x) : v[h] + x;
    }
  __syncthreads();  // red's previous readers are done
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int h = 0; h < H; ++h) red[h][threadIdx.x >> 5] = v[h];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < H; ++h) {
    v[h] = red[h][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v[h] = MAX ? fmaxf(v[h], red[h][w]) : v[h] + red[h][w];
  }
}

constexpr int kHeads = 4;  // heads whose passes run together

// VEC: rows of scores and sums start on 16 bytes.  KEEP: the CTA's scores stay in shared
// memory (where they become e^{s − m}).  chunk: tokens per CTA, a multiple of 4.
template <bool VEC, bool KEEP>
__global__ void __launch_bounds__(kThreads) mass_kernel(const MassArgs a, int chunk, int size) {
  extern __shared__ __align__(16) float sm[];
  float* s_keep = sm;                                              // [group][chunk]
  float* s_ml = sm + (KEEP ? int64_t(a.group) * chunk : 0);        // [group][2]: maximum, sum
  float* s_f = s_ml + 2 * a.group;                                 // [group][2]: row maximum, factor
  __shared__ float red[kHeads][kWarps];
  __shared__ __align__(8) uint64_t s_bar[2];
  __shared__ int s_fail;
  const int tid = threadIdx.x;
  if (tid == 0) {
    s_fail = 0;
    mbarrier_init(smem_addr(&s_bar[0]), 1);
    mbarrier_init(smem_addr(&s_bar[1]), 1);
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
  if constexpr (VEC && KEEP) {
    // the first heads' scores on one barrier, the others' on the next; whole 16 bytes (a
    // row's length is a multiple of 4 tokens, so nothing behind the row is read)
    if (tid == 0 && mine > 0) {
      const uint32_t bytes = uint32_t((mine + 3) / 4 * 16);
      const int early = a.group < kHeads ? a.group : kHeads;
      for (int part = 0; part < 2; ++part) {
        const int h0 = part ? early : 0, h1 = part ? a.group : early;
        if (h0 == h1) continue;
        const uint32_t bar = smem_addr(&s_bar[part]);
        mbarrier_expect_tx(bar, bytes * uint32_t(h1 - h0));
        for (int h = h0; h < h1; ++h) bulk_load(smem_addr(s_keep + int64_t(h) * chunk), sc + int64_t(h) * a.T, bytes, bar);
      }
      if (in) prefetch_l2(in, bytes);
    }
    __syncthreads();
  }

  // ---- each head's maximum over the run, then its sum
  for (int h0 = 0; h0 < a.group; h0 += kHeads) {
    const int hs = a.group - h0 < kHeads ? a.group - h0 : kHeads;
    const float* s = sc + int64_t(h0) * a.T;
    float* k = s_keep + int64_t(h0) * chunk;
    float m[kHeads], l[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) m[h] = -INFINITY, l[h] = 0.f;
    if constexpr (VEC && KEEP) {
      if (mine > 0 && h0 <= kHeads && !mbarrier_wait(smem_addr(&s_bar[h0 ? 1 : 0]), 0)) s_fail = 1;
      for (int t = tid * 4; t < mine; t += kThreads * 4) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if (h >= hs) break;
          float4 v = *reinterpret_cast<const float4*>(k + int64_t(h) * chunk + t);
          if (t + 1 >= mine) v.y = -INFINITY;
          if (t + 2 >= mine) v.z = -INFINITY;
          if (t + 3 >= mine) v.w = -INFINITY;
          m[h] = fmaxf(m[h], fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
        }
      }
    } else {
#pragma unroll 4
      for (int t = tid; t < mine; t += kThreads) {
        float v[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) v[h] = h < hs ? __ldg(s + int64_t(h) * a.T + t) : 0.f;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if (h >= hs) break;
          if constexpr (KEEP) k[int64_t(h) * chunk + t] = v[h];
          m[h] = fmaxf(m[h], v[h]);
        }
      }
    }
    block_reduce<kHeads, true>(m, red);
    if constexpr (VEC && KEEP) {
      for (int t = tid * 4; t < mine; t += kThreads * 4) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if (h >= hs) break;
          const bool some = m[h] != -INFINITY;
          float4* at = reinterpret_cast<float4*>(k + int64_t(h) * chunk + t);
          float4 v = *at;
          v.x = some ? exp2_approx((v.x - m[h]) * kLog2e) : 0.f;
          v.y = some && t + 1 < mine ? exp2_approx((v.y - m[h]) * kLog2e) : 0.f;
          v.z = some && t + 2 < mine ? exp2_approx((v.z - m[h]) * kLog2e) : 0.f;
          v.w = some && t + 3 < mine ? exp2_approx((v.w - m[h]) * kLog2e) : 0.f;
          *at = v;
          l[h] += (v.x + v.y) + (v.z + v.w);
        }
      }
    } else {
      for (int t = tid; t < mine; t += kThreads) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if (h >= hs) break;
          const float v = KEEP ? k[int64_t(h) * chunk + t] : __ldg(s + int64_t(h) * a.T + t);
          const float e = m[h] != -INFINITY ? exp2_approx((v - m[h]) * kLog2e) : 0.f;
          if constexpr (KEEP) k[int64_t(h) * chunk + t] = e;
          l[h] += e;
        }
      }
    }
    block_reduce<kHeads, false>(l, red);
    if (tid < hs) {
      float mm = m[0], ll = l[0];
#pragma unroll
      for (int h = 1; h < kHeads; ++h)
        if (tid == h) mm = m[h], ll = l[h];
      s_ml[2 * (h0 + tid)] = mm;
      s_ml[2 * (h0 + tid) + 1] = s_fail ? __uint_as_float(0x7fc00000u) : ll;  // a copy that never came: NaN
    }
  }
  // ---- the row's maximum and sum; factor = e^{m − row maximum} / row sum
  cluster_sync();
  // (a warp per head, a lane per CTA)
  const int lane = tid & 31;
  for (int h = tid >> 5; h < a.group; h += kWarps) {
    const uint32_t at = smem_addr(s_ml + 2 * h);
    const float mc = lane < size ? __uint_as_float(ld_cluster(at, lane)) : -INFINITY;
    float l = lane < size ? __uint_as_float(ld_cluster(at + 4, lane)) : 0.f, m = mc;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    l = mc == -INFINITY ? 0.f : l * exp2_approx((mc - m) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    if (lane == 0) {
      s_f[2 * h] = m;
      s_f[2 * h + 1] = m == -INFINITY ? 0.f : (KEEP ? exp2_approx((s_ml[2 * h] - m) * kLog2e) : 1.f) / l;
    }
  }
  cluster_sync();  // also: no CTA leaves while its pairs are read
  // ---- the sums
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
  unsigned size = cluster_size(rows, a.T, 512);
  auto share = [&](unsigned c) { return ((a.T + c - 1) / c + 3) / 4 * 4; };
  auto bytes = [&](unsigned c) { return size_t(share(c)) * a.group * 4; };
  // Runs whose scores take more than half of an SM's shared memory leave one CTA per SM.
  // Of clusters above 10 only 7 then run at a time (15 of 9, 11 of 10: the SMs of a GPC),
  // so 10 is tried before 16.
  while (size < 8 && bytes(size) > kMaxScores) size *= 2;
  if (bytes(size) > kMaxScores || (size == 16 && bytes(16) > 100 * 1024)) size = bytes(10) <= kMaxScores ? 10 : 16;
  const int64_t chunk = share(size);
  const bool keep = bytes(size) <= kMaxScores;
  const bool vec = a.T % 4 == 0 && (reinterpret_cast<uintptr_t>(a.scores) | reinterpret_cast<uintptr_t>(a.mass) |
                                    reinterpret_cast<uintptr_t>(a.out)) % 16 == 0;
  const size_t smem = (keep ? size_t(chunk) * a.group : 0) * 4 + size_t(a.group) * 16;
  if (smem > kMaxSmem) return cudaErrorInvalidValue;  // thousands of heads per kv head
  static std::atomic<uint64_t> done[4];
  const int i = (keep ? 2 : 0) + (vec ? 1 : 0);
  auto k = keep ? (vec ? mass_kernel<true, true> : mass_kernel<false, true>)
                : (vec ? mass_kernel<true, false> : mass_kernel<false, false>);
  const cudaError_t e = allow_kernel(k, int(kMaxSmem), &done[i]);
  if (e != cudaSuccess) return e;
  return launch_cluster(k, dim3(unsigned(rows * size)), dim3(kThreads), size, smem, stream, a, int(chunk), int(size));
}

}  // namespace rrq
