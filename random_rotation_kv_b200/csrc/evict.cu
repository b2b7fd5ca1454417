// evict.cu — the tokens of a quantised cache that keep their place, and their rows moved
// together.
//
// Selection: one cluster of up to 16 CTAs per (sequence, kv head); a warp owns a run of 512
// consecutive tokens of its CTA's tile of 8192, 16 per lane, whose masses stay in registers
// (runs of several tiles are read again for every pass).  A key is the mass as an unsigned
// integer of the same order; the sink and the recent tokens have the largest key.  The
// keep-th largest key is found by radix selection: four passes over 8-bit digits from the
// top, each a histogram per CTA (in eight copies by lane: few digits are in use and equal ones
// would queue), the CTAs' histograms summed through distributed shared memory by every
// CTA for itself.  Then every warp counts the keys above and equal to it in its run, the
// counts' prefixes give each kept token its slot, and of the equal ones the first are
// kept; so the order of blocks and atomics never shows in the result.  The passes are bound
// by their four cluster barriers, not by the masses, which are read once.
// Launches overlap, so this kernel may have begun before the one that wrote its inputs ended; every
// load comes after pdl_wait, which makes those writes visible, and none is through the read-only
// path.  What is read once is loaded past L1.
// Moving: a second launch over all SMs copies the rows, 128 per block, 16 bytes (8 where rows
// are not a multiple of 16) per access with the code rows of the new cache written in
// one run; it is bound by memory (2·(d·(kb + vb)/8 + 8) bytes per kept row).
// 131072 tokens x 8 heads to 32768, d = 128, 4-bit: 24 us + 17 us (4.2 TB/s); 24 x 4 heads x 2000
// to 511: 20 us.
#include "cluster.cuh"
#include "evict.h"

namespace rrq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kPer = 16;                      // tokens per lane and tile
constexpr int kTile = kThreads * kPer;        // tokens per tile

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

// REG: a CTA's run is one tile, read once.  Two CTAs per SM: of clusters of 16 with one, only 7
// run at a time (the SMs of a GPC).
template <bool REG>
__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const EvictArgs a, int chunk, int size) {
  __shared__ __align__(16) uint32_t s_copy[256][8];  // [digit][lane mod 8]
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
  // token i of this lane in the tile at `base`: base + first + 32·i
  const int first = warp * (kPer * 32) + lane;
  const int sink = int(a.sink - t0 < 0 ? 0 : a.sink - t0 < chunk ? a.sink - t0 : chunk);  // forced: below it,
  const int64_t tail = n - a.recent - t0;                                                 // and from it on
  const int recent = int(tail < 0 ? 0 : tail < chunk ? tail : chunk);
  float v[kPer];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = base + first + 32 * i;
      v[i] = t < mine ? __ldcg(mass + t) : 0.f;
    }
  };
  auto key_of = [&](int base, int i) {
    const int t = base + first + 32 * i;
    return t < sink || t >= recent ? 0xffffffffu : mass_key(v[i]);
  };
  if constexpr (REG) load(0);
  const int tiles = REG ? 1 : (mine + kTile - 1) / kTile;

  uint32_t prefix = 0, need = uint32_t(a.keep);
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
    reinterpret_cast<uint4*>(s_copy)[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int tile = 0; tile < tiles; ++tile) {
      if constexpr (!REG) load(tile * kTile);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t k = key_of(tile * kTile, i);
        if (tile * kTile + first + 32 * i < mine && (k & mask) == prefix)
          atomicAdd(&s_copy[(k >> shift) & 255u][lane & 7], 1u);
      }
    }
    __syncthreads();
    {
      // two threads per digit
      const uint4 c = reinterpret_cast<const uint4*>(s_copy)[tid];
      uint32_t sum = c.x + c.y + c.z + c.w;
      sum += __shfl_xor_sync(kFull, sum, 1);
      if (!(tid & 1)) s_hist[pass & 1][tid >> 1] = sum;
    }
    cluster_sync();
    {
      // two threads per digit, the even and the odd CTAs
      uint32_t h[8], sum = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int from = 2 * c + (tid & 1);
        h[c] = from < size ? ld_cluster(smem_addr(&s_hist[pass & 1][tid >> 1]), uint32_t(from)) : 0u;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) sum += h[c];
      sum += __shfl_xor_sync(kFull, sum, 1);
      if (!(tid & 1)) s_sum[tid >> 1] = sum;
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
        const uint32_t x = __shfl_down_sync(kFull, suffix, o);
        if (lane + o < 32) suffix += x;
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

  // ---- slots: keys above `prefix`, and the first `need` equal to it, in token order (with
  // several tiles, each tile's warps one after the other)
  uint32_t before_a = 0, before_e = 0;  // of the CTAs before this one
  {
    uint32_t above = 0, equal = 0;
    for (int tile = 0; tile < tiles; ++tile) {
      if constexpr (!REG) load(tile * kTile);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t k = key_of(tile * kTile, i);
        const bool in = tile * kTile + first + 32 * i < mine;
        above += __popc(__ballot_sync(kFull, in && k > prefix));
        equal += __popc(__ballot_sync(kFull, in && k == prefix));
      }
    }
    if (lane == 0) s_warp[0][warp] = above, s_warp[1][warp] = equal;
    __syncthreads();
    if (tid < 2) {
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t x = s_warp[tid][w];
        if (REG) s_warp[tid][w] = sum;  // one tile: the warps' prefixes at once
        sum += x;
      }
      s_count[tid] = sum;
    }
    cluster_sync();
    before_a = __reduce_add_sync(kFull, lane < rank ? ld_cluster(smem_addr(&s_count[0]), uint32_t(lane)) : 0u);
    before_e = __reduce_add_sync(kFull, lane < rank ? ld_cluster(smem_addr(&s_count[1]), uint32_t(lane)) : 0u);
    cluster_arrive();  // this warp has read its counts
  }
  const unsigned below = (1u << lane) - 1u;
  for (int tile = 0; tile < tiles; ++tile) {
    if constexpr (!REG) {
      // this tile's counts per warp
      load(tile * kTile);
      uint32_t above = 0, equal = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t k = key_of(tile * kTile, i);
        const bool in = tile * kTile + first + 32 * i < mine;
        above += __popc(__ballot_sync(kFull, in && k > prefix));
        equal += __popc(__ballot_sync(kFull, in && k == prefix));
      }
      __syncthreads();
      if (lane == 0) s_warp[0][warp] = above, s_warp[1][warp] = equal;
      __syncthreads();
    }
    uint32_t pa = before_a, pe = before_e;
    if constexpr (REG) {
      pa += s_warp[0][warp];
      pe += s_warp[1][warp];
    } else {
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) pa += s_warp[0][w], pe += s_warp[1][w];
        before_a += s_warp[0][w];
        before_e += s_warp[1][w];
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = tile * kTile + first + 32 * i;
      const uint32_t k = key_of(tile * kTile, i);
      const bool in = t < mine;
      const unsigned bg = __ballot_sync(kFull, in && k > prefix), be = __ballot_sync(kFull, in && k == prefix);
      const uint32_t e = pe + __popc(be & below);
      if (in && (k > prefix || (k == prefix && e < need))) {
        const uint32_t slot = pa + __popc(bg & below) + (e < need ? e : need);
        index[slot] = int32_t(t0 + t);
        if (out_mass) out_mass[slot] = v[i];
      }
      pa += __popc(bg);
      pe += __popc(be);
    }
  }
  cluster_wait();  // no CTA leaves while its counts are read
}

// Rows [kept token][kv head] of every sequence, 128 per block and step.  U: bytes per copy.
constexpr int kMoveThreads = 256, kMoveRows = 128;
template <typename U>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  __shared__ int64_t s_src[kMoveRows];
  const int tid = threadIdx.x;
  const int ku = a.k_row / int(sizeof(U)), vu = a.v_row / int(sizeof(U));
  pdl_release();
  pdl_wait();
  for (int64_t b = blockIdx.y; b < a.batch; b += gridDim.y) {
    const int64_t n = clamp_len(a.lens, b, a.cap);
    const int64_t rows = (n < a.keep ? n : a.keep) * a.hkv;  // row s·hkv + g of the new cache
    for (int64_t r0 = int64_t(blockIdx.x) * kMoveRows; r0 < rows; r0 += int64_t(gridDim.x) * kMoveRows) {
      const int live = int(rows - r0 < kMoveRows ? rows - r0 : kMoveRows);
      __syncthreads();  // the previous step has read s_src
      if (tid < live) {
        const int64_t s = (r0 + tid) / a.hkv;
        const int64_t g = (r0 + tid) - s * a.hkv;
        s_src[tid] = (b * a.cap + __ldcg(a.index + (b * a.hkv + g) * a.keep + s)) * a.hkv + g;
      }
      __syncthreads();
      const int64_t to = b * a.keep * a.hkv + r0;
      auto copy = [&](const uint8_t* from, uint8_t* out, int units) {
        const U* f = reinterpret_cast<const U*>(from);
        U* o = reinterpret_cast<U*>(out) + to * units;
        const int total = live * units;
        for (int i0 = tid; i0 < total; i0 += kMoveThreads * 4) {
          U w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned i = unsigned(i0 + e * kMoveThreads);
            if (int(i) < total) w[e] = __ldcg(f + s_src[i / unsigned(units)] * units + i % unsigned(units));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i0 + e * kMoveThreads < total) o[i0 + e * kMoveThreads] = w[e];
        }
      };
      float nu = 0.f;
      const int r = tid & (kMoveRows - 1);
      if (r < live) nu = __ldcg((tid < kMoveRows ? a.k_norms : a.v_norms) + s_src[r]);
      copy(a.k_codes, a.ok_codes, ku);
      copy(a.v_codes, a.ov_codes, vu);
      if (r < live) (tid < kMoveRows ? a.ok_norms : a.ov_norms)[to + r] = nu;
    }
  }
}

template <typename U> cudaError_t launch_move(const EvictArgs& a, cudaStream_t stream) {
  const int64_t most = a.keep < a.cap ? a.keep : a.cap;
  const int64_t blocks = (most * a.hkv + kMoveRows - 1) / kMoveRows;
  const unsigned y = unsigned(a.batch < 65535 ? a.batch : 65535);
  const int64_t fill = (int64_t(kSms) * 16 + y - 1) / y;
  return launch_pdl(evict_move_kernel<U>, dim3(unsigned(blocks < fill ? blocks : fill), y), dim3(kMoveThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t rows = a.batch * a.hkv;
  // runs of one tile where 16 CTAs give them
  unsigned size = cluster_size(rows, a.cap, 512);
  while (size < 16 && (a.cap + size - 1) / size > kTile) size *= 2;
  const int64_t chunk = (a.cap + size - 1) / size;
  const bool reg = chunk <= kTile;
  static std::atomic<uint64_t> done[2];
  auto k = reg ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaError_t e = allow_kernel(k, 0, &done[reg]);
  if (e != cudaSuccess) return e;
  e = launch_cluster(k, dim3(unsigned(rows * size)), dim3(kThreads), size, 0, stream, a, int(chunk), int(size));
  if (e != cudaSuccess) return e;
  return a.k_row % 16 == 0 && a.v_row % 16 == 0 ? launch_move<uint4>(a, stream) : launch_move<uint2>(a, stream);
}

}  // namespace rrq
