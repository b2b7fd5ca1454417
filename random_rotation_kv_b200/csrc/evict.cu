// evict.cu — the tokens of a quantised cache that keep their place, and their rows moved
// together.
//
// Selection: one cluster of up to 16 CTAs per (sequence, kv head), each with a run of
// tokens whose keys it reads once and keeps in shared memory (runs too long for it are
// read again).  A key is the mass as an unsigned integer of the same order; the sink and
// the recent tokens have the largest key.  The keep-th largest key is found by radix
// selection: four passes over 8-bit digits from the top, each a histogram per CTA, the
// CTAs' histograms summed through distributed shared memory by every CTA for itself.
// Then every warp counts the keys above and equal to it in its own run of tokens, the
// counts' prefixes give each kept token its slot, and of the equal ones the first are
// kept; so the order of blocks and atomics never shows in the result.  Moving: a second
// launch over all SMs copies the rows, several per warp, 16 bytes (8 where rows are not a
// multiple of 16) per lane; it is bound by memory (2·(d·(kb + vb)/8 + 8) bytes per kept row).
#include "cluster.cuh"
#include "evict.h"

namespace rrq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int64_t kMaxKeys = 50 * 1024;  // keys a CTA keeps (200 KB)

__device__ __forceinline__ int64_t clamp_len(const int32_t* lens, int64_t b, int64_t cap) {
  if (lens == nullptr) return cap;
  const int64_t n = lens[b];
  return n < 0 ? 0 : n > cap ? cap : n;
}

// Order-preserving key of a mass: NaN lowest (0), −0 as +0.
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <bool KEEP>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a, int chunk, int size) {
  extern __shared__ uint32_t s_keys[];  // [chunk] with KEEP
  __shared__ uint32_t s_hist[2][256];   // alternating passes: the other one may still be read
  __shared__ uint32_t s_sum[256];
  __shared__ uint32_t s_pick[2];        // digit, how many of its keys are kept
  __shared__ uint32_t s_count[2];       // this CTA's keys above and equal
  __shared__ uint32_t s_warp[2][kWarps];
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / size, b = row / a.hkv;
  const int rank = int(blockIdx.x % size);
  const int64_t n = clamp_len(a.lens, b, a.cap);
  const int64_t t0 = int64_t(rank) * chunk;
  const int mine = int(t0 >= n ? 0 : n - t0 < chunk ? n - t0 : chunk);
  const float* mass = a.mass + row * a.cap + t0;
  int32_t* index = a.index + row * a.keep;
  float* out_mass = a.out_mass ? a.out_mass + row * a.keep : nullptr;
  if (row % a.hkv == 0 && rank == 0 && tid == 0) a.out_lens[b] = int32_t(n < a.keep ? n : a.keep);
  if (n <= a.keep) {  // the same in every CTA of the cluster
    for (int t = tid; t < mine; t += kThreads) {
      index[t0 + t] = int32_t(t0 + t);
      if (out_mass) out_mass[t0 + t] = mass[t];
    }
    return;
  }
  auto read_key = [&](int t) {
    return t0 + t < a.sink || t0 + t >= n - a.recent ? 0xffffffffu : mass_key(__ldg(mass + t));
  };
  if constexpr (KEEP) {
#pragma unroll 4
    for (int t = tid; t < mine; t += kThreads) s_keys[t] = read_key(t);
  }
  auto key_at = [&](int t) { return KEEP ? s_keys[t] : read_key(t); };
  for (int i = tid; i < 512; i += kThreads) s_hist[i >> 8][i & 255] = 0;
  __syncthreads();

  uint32_t prefix = 0, need = uint32_t(a.keep);
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
    uint32_t* hist = s_hist[pass & 1];
    for (int t = tid; t - lane < mine; t += kThreads) {
      const uint32_t k = t < mine ? key_at(t) : 0u;
      const bool in = t < mine && (k & mask) == prefix;
      const uint32_t dgt = (k >> shift) & 255u;
      // the first lane's digit is counted once for all that share it: equal masses are common
      const unsigned live = __ballot_sync(kFull, in);
      if (live == 0) continue;
      const int first = __ffs(live) - 1;
      const uint32_t lead = __shfl_sync(kFull, dgt, first);
      const unsigned same = __ballot_sync(kFull, in && dgt == lead);
      if (lane == first) atomicAdd(&hist[dgt], uint32_t(__popc(same)));
      else if (in && !(same >> lane & 1u)) atomicAdd(&hist[dgt], 1u);
    }
    cluster_sync();
    if (tid < 256) {
      uint32_t sum = 0;
      const uint32_t at = smem_addr(&hist[tid]);
      for (int c = 0; c < size; ++c) sum += ld_cluster(at, c);
      s_sum[tid] = sum;
      s_hist[(pass + 1) & 1][tid] = 0;  // its readers met at the barrier above
    }
    __syncthreads();
    if (warp == 0) {
      // lane l: digits [8l, 8l + 8); keys with a larger digit than lane l's
      uint32_t part[8], mysum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mysum += part[i] = s_sum[8 * lane + i];
      uint32_t suffix = mysum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_down_sync(kFull, suffix, o);
        if (lane + o < 32) suffix += v;
      }
      uint32_t above = suffix - mysum;
      if (above < need && need <= suffix) {
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          if (need > above && need <= above + part[i]) {
            s_pick[0] = uint32_t(8 * lane + i);
            s_pick[1] = need - above;
          }
          above += part[i];
        }
      }
    }
    __syncthreads();
    prefix |= s_pick[0] << shift;
    need = s_pick[1];
  }

  // ---- slots: keys above `prefix`, and the first `need` equal to it, in token order.
  // Warp w: tokens [w·run, (w + 1)·run) of this CTA's.
  const int run = (mine + kThreads - 1) / kThreads * 32;
  const int w0 = warp * run, w1 = w0 + run < mine ? w0 + run : mine;
  uint32_t above = 0, equal = 0;
  for (int t = w0; t < w1; t += 32) {
    const bool in = t + lane < w1;
    const uint32_t k = in ? key_at(t + lane) : 0u;
    above += __popc(__ballot_sync(kFull, in && k > prefix));
    equal += __popc(__ballot_sync(kFull, in && k == prefix));
  }
  if (lane == 0) s_warp[0][warp] = above, s_warp[1][warp] = equal;
  __syncthreads();
  if (tid < 2) {
    uint32_t sum = 0;
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t v = s_warp[tid][w];
      s_warp[tid][w] = sum;
      sum += v;
    }
    s_count[tid] = sum;
  }
  cluster_sync();
  uint32_t pa = s_warp[0][warp], pe = s_warp[1][warp];
  for (int c = 0; c < rank; ++c) {
    pa += ld_cluster(smem_addr(&s_count[0]), c);
    pe += ld_cluster(smem_addr(&s_count[1]), c);
  }
  const unsigned below = (1u << lane) - 1u;
  for (int t = w0; t < w1; t += 32) {
    const bool in = t + lane < w1;
    const uint32_t k = in ? key_at(t + lane) : 0u;
    const unsigned bg = __ballot_sync(kFull, in && k > prefix), be = __ballot_sync(kFull, in && k == prefix);
    const uint32_t e = pe + __popc(be & below);
    if (in && (k > prefix || (k == prefix && e < need))) {
      const uint32_t slot = pa + __popc(bg & below) + (e < need ? e : need);
      index[slot] = int32_t(t0 + t + lane);
      if (out_mass) out_mass[slot] = mass[t + lane];
    }
    pa += __popc(bg);
    pe += __popc(be);
  }
  cluster_sync();  // no CTA leaves while its counts are read
}

// Rows [kept token][kv head] of every sequence.  U: bytes per copy; `lanes` (a power of two)
// lanes per row, kRows rows per group of lanes with their loads in flight together.
template <typename U>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a, int log2l) {
  constexpr int kRows = 4;
  const int tid = threadIdx.x, lanes = 1 << log2l, sub = tid & (lanes - 1);
  const int ku = a.k_row / int(sizeof(U)), vu = a.v_row / int(sizeof(U));
  const int per = 256 >> log2l;  // rows per block and step
  pdl_release();
  pdl_wait();
  for (int64_t b = blockIdx.y; b < a.batch; b += gridDim.y) {
    const int64_t n = clamp_len(a.lens, b, a.cap);
    const int64_t rows = (n < a.keep ? n : a.keep) * a.hkv;  // row s·hkv + g of the new cache
    for (int64_t r0 = int64_t(blockIdx.x) * (per * kRows) + (tid >> log2l); r0 < rows; r0 += int64_t(gridDim.x) * (per * kRows)) {
      int64_t src[kRows];
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        const int64_t r = r0 + e * per;
        src[e] = -1;
        if (r < rows) {
          const int64_t s = r / a.hkv;
          const int g = int(r - s * a.hkv);
          src[e] = (b * a.cap + __ldg(a.index + (b * a.hkv + g) * a.keep + s)) * a.hkv + g;
        }
      }
      for (int i = sub; i < ku + vu + 2; i += lanes) {
        const bool norm = i >= ku + vu;
        U w[kRows];
        float f[kRows];
#pragma unroll
        for (int e = 0; e < kRows; ++e)
          if (src[e] >= 0) {
            if (norm) f[e] = __ldg((i == ku + vu ? a.k_norms : a.v_norms) + src[e]);
            else if (i < ku) w[e] = __ldg(reinterpret_cast<const U*>(a.k_codes + src[e] * a.k_row) + i);
            else w[e] = __ldg(reinterpret_cast<const U*>(a.v_codes + src[e] * a.v_row) + (i - ku));
          }
#pragma unroll
        for (int e = 0; e < kRows; ++e)
          if (src[e] >= 0) {
            const int64_t r = b * a.keep * a.hkv + r0 + e * per;
            if (norm) (i == ku + vu ? a.ok_norms : a.ov_norms)[r] = f[e];
            else if (i < ku) reinterpret_cast<U*>(a.ok_codes + r * a.k_row)[i] = w[e];
            else reinterpret_cast<U*>(a.ov_codes + r * a.v_row)[i - ku] = w[e];
          }
      }
    }
  }
}

template <typename U> cudaError_t launch_move(const EvictArgs& a, cudaStream_t stream) {
  const int units = (a.k_row + a.v_row) / int(sizeof(U)) + 2;
  int log2l = 2;
  while (log2l < 5 && (1 << log2l) < units) ++log2l;
  const int64_t most = a.keep < a.cap ? a.keep : a.cap;
  const int64_t blocks = (most * a.hkv + (1024 >> log2l) - 1) / (1024 >> log2l);
  const unsigned y = unsigned(a.batch < 65535 ? a.batch : 65535);
  const int64_t fill = (int64_t(148) * 8 + y - 1) / y;
  auto k = evict_move_kernel<U>;
  return launch_pdl(k, dim3(unsigned(blocks < fill ? blocks : fill), y), dim3(256), 0, stream, a, log2l);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t rows = a.batch * a.hkv;
  unsigned size = cluster_size(rows, a.cap, 512);
  while (size < 16 && (a.cap + size - 1) / size > kMaxKeys) size *= 2;
  const int64_t chunk = (a.cap + size - 1) / size;
  const bool keep = chunk <= kMaxKeys;
  const cudaError_t e = launch_cluster(keep ? evict_select_kernel<true> : evict_select_kernel<false>,
                                       dim3(unsigned(rows * size)), dim3(kThreads), size, keep ? size_t(chunk) * 4 : 0,
                                       stream, a, int(chunk), int(size));
  if (e != cudaSuccess) return e;
  return a.k_row % 16 == 0 && a.v_row % 16 == 0 ? launch_move<uint4>(a, stream) : launch_move<uint2>(a, stream);
}

}  // namespace rrq
