// evict.cu — the tokens of a quantised cache that keep their place, and their rows moved
// together.
//
// Selection per (sequence, kv head): the keep-th largest of n keys by radix selection
// (four passes over 8-bit digits, a histogram each), then one pass in token order that
// keeps every key above it and the first of those equal to it.  A key is the mass as
// an unsigned integer of the same order; the sink and the recent tokens have the
// largest key.  Then the rows are copied, one slot of one kv head after the other.
#include "evict.h"
#include "rrq_device.cuh"

namespace rrq {
namespace {

constexpr int kThreads = 1024;

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

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ unsigned hist[256];
  __shared__ unsigned s_prefix, s_need;
  __shared__ unsigned s_above[32], s_equal[32];
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x, b = row / a.hkv;
  const int64_t n = clamp_len(a.lens, b, a.cap);
  const float* mass = a.mass + row * a.cap;
  int32_t* index = a.index + row * a.keep;
  if (row % a.hkv == 0 && tid == 0) a.out_lens[b] = int32_t(n < a.keep ? n : a.keep);
  if (n <= a.keep) {
    for (int64_t t = tid; t < n; t += kThreads) {
      index[t] = int32_t(t);
      if (a.out_mass) a.out_mass[row * a.keep + t] = mass[t];
    }
    return;
  }
  auto key_at = [&](int64_t t) {
    return t < a.sink || t >= n - a.recent ? 0xffffffffu : mass_key(mass[t]);
  };
  // the keep-th largest key: digits from the top; s_need = how many of the keys with
  // the digits found so far belong to the kept ones
  uint32_t prefix = 0, need = uint32_t(a.keep);
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int64_t t = tid; t < n; t += kThreads) {
      const uint32_t k = key_at(t);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = need;
      int dgt = 255;
      while (dgt > 0 && hist[dgt] < left) left -= hist[dgt--];
      s_prefix = prefix | (uint32_t(dgt) << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }
  // in token order: keys above `prefix`, and the first `need` equal to it
  uint32_t above = 0, equal = 0;  // tokens so far
  for (int64_t t0 = 0; t0 < n; t0 += kThreads) {
    const int64_t t = t0 + tid;
    const uint32_t k = t < n ? key_at(t) : 0u;
    const bool gt = t < n && k > prefix, eq = t < n && k == prefix;
    const unsigned bg = __ballot_sync(kFull, gt), be = __ballot_sync(kFull, eq);
    if (lane == 0) { s_above[warp] = __popc(bg); s_equal[warp] = __popc(be); }
    __syncthreads();
    uint32_t pa = above, pe = equal, ta = 0, te = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) { pa += ta; pe += te; }
      ta += s_above[w];
      te += s_equal[w];
    }
    const unsigned below = (1u << lane) - 1u;
    pa += __popc(bg & below);
    pe += __popc(be & below);
    if (gt || (eq && pe < need)) {
      const uint32_t slot = pa + (pe < need ? pe : need);
      index[slot] = int32_t(t);
      if (a.out_mass) a.out_mass[row * a.keep + slot] = mass[t];
    }
    above += ta;
    equal += te;
    __syncthreads();
  }
}

// One warp per kept row: its code bytes (8 at a time) and its norms.
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.batch * a.keep * a.hkv;
  const int64_t step = int64_t(gridDim.x) * 8;
  for (int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); r < rows; r += step) {
    const int64_t b = r / (a.keep * a.hkv), s = r / a.hkv % a.keep, g = r % a.hkv;
    const int64_t n = clamp_len(a.lens, b, a.cap);
    if (s >= n) continue;
    const int64_t src = (b * a.cap + a.index[(b * a.hkv + g) * a.keep + s]) * a.hkv + g;
    for (int i = lane * 8; i < a.k_row; i += 256)
      *reinterpret_cast<uint2*>(a.ok_codes + r * a.k_row + i) =
          *reinterpret_cast<const uint2*>(a.k_codes + src * a.k_row + i);
    for (int i = lane * 8; i < a.v_row; i += 256)
      *reinterpret_cast<uint2*>(a.ov_codes + r * a.v_row + i) =
          *reinterpret_cast<const uint2*>(a.v_codes + src * a.v_row + i);
    if (lane == 0) a.ok_norms[r] = a.k_norms[src];
    if (lane == 1) a.ov_norms[r] = a.v_norms[src];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(unsigned(a.batch * a.hkv)), dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  const int grid = grid_for(reinterpret_cast<const void*>(evict_move_kernel), 256, 0,
                            (a.batch * a.keep * a.hkv + 7) / 8);
  return launch_pdl(evict_move_kernel, grid, 256, 0, stream, a);
}

}  // namespace rrq
