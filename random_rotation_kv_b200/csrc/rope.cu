// rope.cu — rotary positions: every pair of coordinates of a vector turned by its
// token's angle.
//
// (a', b') = factor·(a·cos φ − b·sin φ, a·sin φ + b·cos φ), φ = p·θ_i.  The angle is
// needed modulo one turn only, so θ_i comes as the 64-bit fraction θ_i/2π·2^64, rounded, and
// p·θ_i is one wrapping 64-bit product: within |p|·2^-65 turns for every int64 position, where an
// fp32 product would lose all digits of φ from p ≈ 10^6 on.  Its top 32 bits (cut: 2^-32 turns or
// 1.5e-9 more) are split into the nearest quarter turn (which swaps and negates) and a
// remainder of at most an eighth of a turn, whose sine and cosine are taken in fp32.
//
// Bound by memory: x is read once and y written once.  A thread owns eight pairs of one
// token (two runs of 8 coordinates, or one of 16) and walks heads with them, so a sine and
// cosine serve every head the thread walks; the heads are spread over more threads only
// while there are too few tokens to fill the GPU.  Pairs that do not come in eights
// (rot not a multiple of 16) and addresses off 32 bytes take one pair per thread.
// 32768 x 8 x 128 fp16: 22-24 us, 5.6-6.0 TB/s; with 90 or 40 of the 128 coordinates turned (one pair
// per thread, bound by the number of its 2-byte accesses) 70 and 65 us; one token of 32 heads: 1.8 us.
#include <cstring>

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

// 16 consecutive bytes (W = 4) or 32 (W = 8) as 32-bit words.  Plain accesses: y may be x.
template <int W> __device__ __forceinline__ void ld_words(const void* p, uint32_t (&w)[W]) {
  if constexpr (W == 8)
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  else
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p)
                 : "memory");
}
template <int W> __device__ __forceinline__ void st_words(void* p, const uint32_t (&w)[W]) {
  if constexpr (W == 8)
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  else
    asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
// Eight elements in 4 or 8 words.
template <typename T, int W> __device__ __forceinline__ void to_float(const uint32_t (&w)[W], float (&v)[8]) {
  if constexpr (W == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(w[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <typename T, int W> __device__ __forceinline__ void from_float(const float (&v)[8], uint32_t (&w)[W]) {
  if constexpr (W == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<T>(make_float2(v[2 * i], v[2 * i + 1]));
  }
}

// One thread per (token, 16 coordinates, block of `per` heads): eight pairs, or 16 copied
// coordinates from rot on.  log2u: log2(d / 16) threads per token.
template <typename T, bool INTER, int N>
__global__ void __launch_bounds__(kThreads) rope8_kernel(const RopeArgs a, const __grid_constant__ RopeTurns<N> f, int log2u,
                                                         int per) {
  constexpr int W = 8 * Elem<T>::kBytes / 4;  // words of eight elements
  __shared__ uint64_t s_turns[N];
  pdl_release();
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < half; i += kThreads) s_turns[i] = f.turns[i];
  __syncthreads();
  pdl_wait();
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int u = int(i) & ((1 << log2u) - 1);
  const int64_t t = i >> log2u;
  if (t >= a.n) return;
  const int h0 = blockIdx.y * per, h1 = h0 + per < a.heads ? h0 + per : a.heads;
  const bool turn = u * 16 < a.rot;
  // the two runs of eight: pairs [8u, 8u + 8), or coordinates [16u, 16u + 16)
  const int c0 = INTER || !turn ? 16 * u : 8 * u, c1 = INTER || !turn ? c0 + 8 : c0 + half;
  const int64_t base = (t * a.heads + h0) * a.d;
  const T* x = static_cast<const T*>(a.x) + base;
  T* y = static_cast<T*>(a.y) + base;
  if (!turn && a.x == a.y) return;
  float2 cs[8];
  if (turn) {
    const int64_t pos = a.positions[t];
#pragma unroll
    for (int k = 0; k < 8; ++k) cs[k] = turn_of(s_turns[8 * u + k], pos, a.cos_factor, a.sin_factor);
  }
  // the same loads and stores for turned and copied runs, whose threads share warps
  constexpr int kAhead = W == 8 ? 2 : 4;  // heads whose loads are in flight together
  for (int h = h0; h < h1; h += kAhead, x += kAhead * a.d, y += kAhead * a.d) {
    uint32_t p[kAhead][W], q[kAhead][W];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (h + e < h1) {
        ld_words(x + e * a.d + c0, p[e]);
        ld_words(x + e * a.d + c1, q[e]);
      }
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (h + e < h1) {
        if (turn) {
          float v0[8], v1[8];
          to_float<T, W>(p[e], v0);
          to_float<T, W>(q[e], v1);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float& va = INTER ? (k < 4 ? v0[2 * k] : v1[2 * k - 8]) : v0[k];
            float& vb = INTER ? (k < 4 ? v0[2 * k + 1] : v1[2 * k - 7]) : v1[k];
            const float r = va * cs[k].x - vb * cs[k].y;
            vb = va * cs[k].y + vb * cs[k].x;
            va = r;
          }
          from_float<T, W>(v0, p[e]);
          from_float<T, W>(v1, q[e]);
        }
        st_words(y + e * a.d + c0, p[e]);
        st_words(y + e * a.d + c1, q[e]);
      }
  }
}

// One thread per (token, pair or copied coordinate, block of heads).
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, const __grid_constant__ RopeTurns<N> f, int hblocks) {
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
    const float2 cs = turn_of(f.turns[u], a.positions[t], a.cos_factor, a.sin_factor);
    const int ia = a.interleaved ? 2 * u : u, ib = a.interleaved ? 2 * u + 1 : u + half;
    for (int h = h0; h < h1; ++h) {
      const float p = float(x[int64_t(h) * a.d + ia]), q = float(x[int64_t(h) * a.d + ib]);
      y[int64_t(h) * a.d + ia] = T(p * cs.x - q * cs.y);
      y[int64_t(h) * a.d + ib] = T(p * cs.y + q * cs.x);
    }
  }
}

// Blocks of heads: one while the tokens alone give every SM 1536 threads.  All heads in one thread:
// a token of 32 heads x 128 5.8 us against 1.8, 64 tokens 8.1 against 2.3; 32768 tokens x 8
// heads 22.4 us against 24.0 with two blocks.
int head_blocks(int64_t threads, int heads) {
  const int64_t want = int64_t(kSms) * 1536;
  const int64_t hb = (want + threads - 1) / threads;
  return int(hb < heads ? hb : heads);
}

template <typename T, int N> cudaError_t launch_pairs(const RopeArgs& a, const RopeTurns<N>& f, cudaStream_t stream) {
  const bool wide = a.rot % 16 == 0 && (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) % 32 == 0;
  if (wide && a.n * (a.d / 16) < (int64_t(1) << 38)) {
    int log2u = 2;
    while (16 << log2u < a.d) ++log2u;
    const int64_t threads = a.n << log2u;
    int hb = head_blocks(threads, a.heads);
    if (hb > 65535) hb = 65535;
    const int per = (a.heads + hb - 1) / hb;
    const dim3 grid(unsigned((threads + kThreads - 1) / kThreads), unsigned((a.heads + per - 1) / per));
    return launch_pdl(a.interleaved ? rope8_kernel<T, true, N> : rope8_kernel<T, false, N>, grid, dim3(kThreads), 0, stream,
                      a, f, log2u, per);
  }
  const int units = a.rot / 2 + (a.d - a.rot);
  const int hb = head_blocks(a.n * units, a.heads);
  const int64_t blocks = (a.n * hb * units + kThreads - 1) / kThreads;
  const int grid = grid_for(reinterpret_cast<const void*>(rope_kernel<T, N>), kThreads, 0, blocks);
  return launch_pdl(rope_kernel<T, N>, grid, kThreads, 0, stream, a, f, hb);
}

template <typename T>
cudaError_t launch_typed(const RopeArgs& a, const RopeTurns<kRopeMaxPairs>& f, cudaStream_t stream) {
  if (a.rot > 128) return launch_pairs<T>(a, f, stream);
  RopeTurns<64> few;
  std::memcpy(&few, &f, sizeof(few));
  return launch_pairs<T>(a, few, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, const RopeTurns<kRopeMaxPairs>& f, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case RRQ_F16: return launch_typed<__half>(a, f, stream);
    case RRQ_BF16: return launch_typed<__nv_bfloat16>(a, f, stream);
    default: return launch_typed<float>(a, f, stream);
  }
}

}  // namespace rrq
