// rope.cu — rotary positions: every pair of coordinates of a vector turned by its
// token's angle.
//
// (a', b') = factor·(a·cos φ − b·sin φ, a·sin φ + b·cos φ), φ = p·θ_i.  The angle is
// needed modulo one turn only, so θ_i comes as the 64-bit fraction θ_i/2π·2^64 and
// p·θ_i is one wrapping 64-bit product: exact for every int64 position, where an
// fp32 product would lose all digits of φ from p ≈ 10^6 on.  The top 32 bits are split
// into the nearest quarter turn (which swaps and negates) and a remainder of at most
// an eighth of a turn, whose sine and cosine are taken in fp32.
//
// Bound by memory: x is read once and y written once.  A thread owns one block of
// pairs of one token and walks heads with it, so a sine and cosine serve every head
// the thread walks; the heads are spread over more threads only while there are too few
// tokens to fill the GPU.
#include "rope.h"
#include "rrq_device.cuh"

namespace rrq {
namespace {

constexpr int kThreads = 256;

// cos and sin of pair i at position p, times the factors.
__device__ __forceinline__ float2 turn_of(uint64_t turns, int64_t p, float cf, float sf) {
  const uint32_t t = uint32_t((uint64_t(p) * turns) >> 32);  // 2^-32 turns
  const uint32_t quarter = (t + 0x20000000u) >> 30;          // nearest quarter turn
  const int32_t r = int32_t(t - (quarter << 30));            // within ± an eighth of a turn
  float s, c;
  sincospif(float(r) * 0x1p-31f, &s, &c);  // half turns
  const float cs = quarter & 1u ? s : c, sn = quarter & 1u ? c : s;
  const float cq = ((quarter + 1u) & 2u) ? -cs : cs;  // quarters 1 and 2: cos negative
  const float sq = (quarter & 2u) ? -sn : sn;         // quarters 2 and 3: sin negative
  return make_float2(cq * cf, sq * sf);
}

template <typename T> __device__ __forceinline__ float to_f(T v) { return float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v) { return T(v); }

// One thread per (token, pair, block of heads); plain element accesses.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int hblocks) {
  pdl_release();
  pdl_wait();
  const int half = a.rot / 2, units = half + (a.d - a.rot);  // pairs, then copied coordinates
  const int64_t total = a.n * hblocks * units;
  const int per = (a.heads + hblocks - 1) / hblocks;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total; i += int64_t(gridDim.x) * kThreads) {
    const int u = int(i % units);
    const int64_t th = i / units;
    const int64_t t = th / hblocks;
    const int h0 = int(th % hblocks) * per, h1 = h0 + per < a.heads ? h0 + per : a.heads;
    const T* x = static_cast<const T*>(a.x) + t * a.heads * a.d;
    T* y = static_cast<T*>(a.y) + t * a.heads * a.d;
    if (u >= half) {
      const int c = a.rot + (u - half);
      for (int h = h0; h < h1; ++h) y[int64_t(h) * a.d + c] = x[int64_t(h) * a.d + c];
      continue;
    }
    const float2 cs = turn_of(a.turns[u], a.positions[t], a.cos_factor, a.sin_factor);
    const int ia = a.interleaved ? 2 * u : u, ib = a.interleaved ? 2 * u + 1 : u + half;
    for (int h = h0; h < h1; ++h) {
      const float p = to_f(x[int64_t(h) * a.d + ia]), q = to_f(x[int64_t(h) * a.d + ib]);
      y[int64_t(h) * a.d + ia] = from_f<T>(p * cs.x - q * cs.y);
      y[int64_t(h) * a.d + ib] = from_f<T>(p * cs.y + q * cs.x);
    }
  }
}

template <typename T> cudaError_t launch_typed(const RopeArgs& a, cudaStream_t stream) {
  const int units = a.rot / 2 + (a.d - a.rot);
  const int64_t want = int64_t(148) * 2048;
  int64_t hb = (want + a.n * units - 1) / (a.n * units);
  if (hb > a.heads) hb = a.heads;
  const int64_t blocks = (a.n * hb * units + kThreads - 1) / kThreads;
  const int grid = grid_for(reinterpret_cast<const void*>(rope_kernel<T>), kThreads, 0, blocks);
  return launch_pdl(rope_kernel<T>, grid, kThreads, 0, stream, a, int(hb));
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case RRQ_F16: return launch_typed<__half>(a, stream);
    case RRQ_BF16: return launch_typed<__nv_bfloat16>(a, stream);
    default: return launch_typed<float>(a, stream);
  }
}

}  // namespace rrq
