// attention_shared_tc.cu — partial states of attention over a quantised cache on the
// 5th-generation tensor cores, for head sizes up to 256: up to 128 query rows against a
// run of tiles of one kv head (attention_shared.h).
//
// With the rows' rotated queries q' (fp16, a power of two 2^-e per row taken out; for
// fp16 queries at d ≤ 128 a second fp16 part holds what the first rounds off) and the
// levels c as fp16,
//     S = Q'·C_Kᵀ,   x = 2^e·ν^K_t·S,   P = 2^{x − m'}·ν^V_t,   O += P·C_V,
// where m' follows the row's running maximum m: it moves only when m grows by more than
// 4 (powers of two), so O is rarely rescaled, and it carries the power of two that
// brings the weights into fp16's range: with N the power of two below the largest ν^V
// seen (it moves when that grows fourfold), m' = m − 8 + log2 N, so weights are at most
// 2^15 and keep full precision down to 2^-22 of the largest.  The state (m', Σ 2^{x − m'}, O)
// is what the merge takes.
//
// One CTA per SM walks its range of tiles (128 tokens, 64 for d = 256), 13 warps:
//  * warps 4–11 read the packed codes one tile ahead into registers, turn code pairs into
//    level pairs by one shared-memory lookup per byte (tables of 256 pairs, one copy per
//    lane so that no bank conflicts; a value byte holds one coordinate of two tokens, so
//    V is laid out transposed without a transposition) and write K [token][coordinate] and
//    V [coordinate][token] as fp16 in the 128-byte swizzle, two stages each;
//  * warp 12 issues the products: S from the queries in tensor memory and K, O from the
//    weights in tensor memory and V; the next tile's S runs while this tile's weights
//    are made;
//  * warps 0–3 own one query row per thread: S from tensor memory, maximum, weights back
//    into S's own columns as fp16, sums in registers.
// Tensor memory: S twice, O and the queries (all of its 512 columns at d = 256).
// Every wait is bounded; a wait that gives up makes the CTA's states NaN.
#include "attention_shared.cuh"
#include "tcgen05.cuh"

namespace rrq {
namespace {

constexpr uint32_t kWaitLimit = 1u << 24;  // polls, a few seconds in all
constexpr int kSoftWarps = 4, kFillWarps = 8, kFill = kFillWarps * 32;
constexpr int kThreads = (kSoftWarps + kFillWarps + 1) * 32;

template <int D> struct Tc {
  static constexpr int TN = D <= 128 ? 128 : 64;     // tokens per tile
  static constexpr int OCT = D / 8 * TN / kFill;     // K octets per filling thread
  static constexpr uint32_t TILE = TN * D * 2;       // bytes of a K or V stage
  // shared addresses (the dynamic base is checked to be kBase)
  static constexpr uint32_t kBase = 0x400;
  static constexpr uint32_t BARS = 0x400;
  static constexpr uint32_t TSLOT = 0x4C0;
  static constexpr uint32_t FAIL = 0x4D0;
  static constexpr uint32_t VMAX = 0x500;            // [4 tiles][4 warps] largest value norm
  static constexpr uint32_t NK = 0x800, NV = 0x1000; // [4 tiles][TN] norms
  static constexpr uint32_t K1 = 0x8000;             // K stage 1
  static constexpr uint32_t TABLE = 0x10000;         // K pairs at +0, V pairs at +128 of every 256 bytes
  static constexpr uint32_t K0 = 0x20000;
  static constexpr uint32_t V0 = 0x28000;            // V stages
  static constexpr size_t kTotal = 0x38000 - kBase;
  // tensor memory columns
  static constexpr int S = 0, O = 2 * TN, Q = O + D, QL = Q + D / 2;
  static constexpr uint32_t idesc(int n) { return (1u << 4) | (uint32_t(n / 8) << 17) | ((128u / 16) << 24); }
  static_assert(NV + 4 * TN * 4 <= 0x8000 && TILE <= 0x8000 && V0 + 2 * 0x8000 <= kBase + 227 * 1024, "layout");
};

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* fail) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *fail) return false;
  }
  *fail = 1;
  return false;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D[tmem] (+)= A[tmem]·B, kind::f16, one CTA.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ---- the filling warps' reads and writes, by code width
// Words of a K row that hold OCT octets, in loads as wide as their alignment allows.
template <int B, int OCT> __device__ __forceinline__ void load_k(const uint8_t* p, uint32_t (&w)[8]) {
  constexpr int W = OCT * B / 4;
  if constexpr (W % 4 == 0) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (W % 2 == 0) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + i);
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  }
}
// Octet i of those words as nibbles.
template <int B> __device__ __forceinline__ uint32_t octet_of(const uint32_t (&w)[8], int i) {
  if constexpr (B == 4) return w[i];
  const int bit = 8 * B * i, k = bit >> 5, sh = bit & 31;
  uint32_t v = w[k] >> sh;
  if (sh + 8 * B > 32) v = __funnelshift_r(w[k], w[k + 1 < 8 ? k + 1 : 7], sh);
  return octet_nibbles(v & (B == 3 ? 0xffffffu : B == 2 ? 0xffffu : 0xffu), B);
}
// The B bytes of octet o of 8 rows (3-bit octets as the two words they may touch).
template <int B>
__device__ __forceinline__ void load_v(const uint8_t* const (&p)[8], int o, uint32_t (&w)[16]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if constexpr (B == 4) w[r] = __ldg(reinterpret_cast<const uint32_t*>(p[r]) + o);
    else if constexpr (B == 2) w[r] = __ldg(reinterpret_cast<const uint16_t*>(p[r]) + o);
    else if constexpr (B == 1) w[r] = __ldg(p[r] + o);
    else {
      w[r] = __ldg(reinterpret_cast<const uint32_t*>(p[r]) + (3 * o) / 4);
      w[8 + r] = __ldg(reinterpret_cast<const uint32_t*>(p[r]) + (3 * o + 2) / 4);
    }
  }
}

// Level pair of byte k of `w`; `lane_word` = table | copy of the lane.
template <int K> __device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t lane_word) {
  return lds_u32(__byte_perm(w, lane_word, K == 0 ? 0x7604u : K == 1 ? 0x7614u : K == 2 ? 0x7624u : 0x7634u));
}

template <int B, int OCT>
__device__ __forceinline__ void put_k(const uint32_t (&w)[8], uint32_t row, int c0, int tok, uint32_t lane_word) {
#pragma unroll
  for (int i = 0; i < OCT; ++i) {
    const uint32_t n = octet_of<B>(w, i);
    sts_v4(row + (uint32_t((c0 + i) ^ (tok & 7)) << 4), pair_of<0>(n, lane_word), pair_of<1>(n, lane_word),
           pair_of<2>(n, lane_word), pair_of<3>(n, lane_word));
  }
}
template <int B>
__device__ __forceinline__ void put_v(const uint32_t (&w)[16], int o, uint32_t row, int kb, uint32_t lane_word) {
  uint32_t n[8], ev[4], od[4];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if constexpr (B == 4) n[r] = w[r];
    else if constexpr (B == 3) n[r] = octet_nibbles(__funnelshift_r(w[r], w[8 + r], 8 * ((3 * o) & 3)) & 0xffffffu, 3);
    else n[r] = octet_nibbles(w[r], B);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t a = n[2 * q], b = n[2 * q + 1];
    ev[q] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);  // coordinates 0, 2, 4, 6 of two tokens
    od[q] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);  // 1, 3, 5, 7
  }
  auto put = [&](int i, auto k, const uint32_t (&e)[4]) {
    constexpr int K = decltype(k)::value;
    sts_v4(row + uint32_t(i) * 128 + (uint32_t(kb ^ i) << 4), pair_of<K>(e[0], lane_word), pair_of<K>(e[1], lane_word),
           pair_of<K>(e[2], lane_word), pair_of<K>(e[3], lane_word));
  };
  put(0, std::integral_constant<int, 0>{}, ev);
  put(1, std::integral_constant<int, 0>{}, od);
  put(2, std::integral_constant<int, 1>{}, ev);
  put(3, std::integral_constant<int, 1>{}, od);
  put(4, std::integral_constant<int, 2>{}, ev);
  put(5, std::integral_constant<int, 2>{}, od);
  put(6, std::integral_constant<int, 3>{}, ev);
  put(7, std::integral_constant<int, 3>{}, od);
}

// Position in a range, one tile at a time.
struct Cursor {
  int range, pos, end, i;
  Segment s;
  __device__ __forceinline__ Cursor(const SharedArgs& a, int r) : range(r), i(0) {
    const int64_t start = int64_t(r) * a.head[1];
    const int total = a.head[0];
    pos = int(start < total ? start : total);
    end = int(start + a.head[1] < total ? start + a.head[1] : total);
    if (pos < end) s = segment_at(a, range, pos, end);
  }
  __device__ __forceinline__ bool live() const { return pos < end; }
  __device__ __forceinline__ void next(const SharedArgs& a) {
    if (++i == s.tiles) {
      pos += s.tiles;
      i = 0;
      if (pos < end) s = segment_at(a, range, pos, end);
    }
  }
};

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ SharedArgs a) {
  using L = Tc<D>;
  constexpr int TN = L::TN;
  extern __shared__ __align__(1024) uint8_t dsm[];
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int range = blockIdx.x;
  auto at = [&](uint32_t addr) { return dsm + (addr - L::kBase); };
  uint64_t* bars = reinterpret_cast<uint64_t*>(at(L::BARS));
  uint64_t* q_full = bars;
  auto k_full = [&](int j) { return &bars[1 + (j & 1)]; };
  auto v_full = [&](int j) { return &bars[3 + (j & 1)]; };
  auto s_full = [&](int j) { return &bars[5 + (j & 1)]; };
  auto p_full = [&](int j) { return &bars[7 + (j & 1)]; };
  auto o_done = [&](int j) { return &bars[9 + (j & 1)]; };
  auto phase = [](int j) { return uint32_t(j >> 1) & 1u; };
  uint32_t* tslot = reinterpret_cast<uint32_t*>(at(L::TSLOT));
  volatile int* fail = reinterpret_cast<volatile int*>(at(L::FAIL));
  const bool placed = smem_addr(dsm) == L::kBase;  // the launch checks it too

  if (tid == 0) {
    mbar_init(q_full, kSoftWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), kFillWarps);
      mbar_init(v_full(s), kFillWarps);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), kSoftWarps);
      mbar_init(o_done(s), 1);
    }
    *fail = placed ? 0 : 1;
    fence_mbarrier_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // entry b of the tables: the levels of its low and its high nibble
  for (int i = tid; i < 256 * 64 && placed; i += kThreads) {
    const int b = i >> 6;
    const float* lev = i & 32 ? a.v_levels : a.k_levels;
    const float f = i & 32 ? a.v_alpha : a.k_alpha;
    const __half2 h = __floats2half2_rn(lev[b & 15] * f, lev[b >> 4] * f);
    *reinterpret_cast<__half2*>(at(L::TABLE + uint32_t(b) * 256 + uint32_t(i & 63) * 4)) = h;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();  // from here on, global memory

  if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- softmax: thread = query row
    const uint32_t tl = tmem + (uint32_t(32 * warp) << 16);
    Cursor c(a, range);
    int j = 0;
    while (c.live()) {
      const Segment& s = c.s;
      const bool row_ok = tid < s.nrows, warp_ok = 32 * warp < s.nrows;
      const int64_t qrow = int64_t(s.g) * a.rows + s.row0 + (row_ok ? tid : 0);
      bool ok = *fail == 0;
      float rs = 1.f;
      if (warp_ok) {
        rs = a.qexp[qrow];
#pragma unroll
        for (int part = 0; part < (SPLIT ? 2 : 1); ++part) {
          const uint4* q = reinterpret_cast<const uint4*>((part ? a.ql : a.qh) + qrow * D);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t r[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 v = __ldcg(q + 4 * i + k);
              r[4 * k] = v.x, r[4 * k + 1] = v.y, r[4 * k + 2] = v.z, r[4 * k + 3] = v.w;
            }
            tmem_st16(tl + uint32_t((part ? L::QL : L::Q) + 16 * i), r);
          }
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      float m = 0.f, mp = 0.f, vn = 0.f;  // running maximum, m', N
      float2 l2 = make_float2(0.f, 0.f);
      for (int i = 0; i < s.tiles; ++i, ++j) {
        ok = ok && wait_for(s_full(j), phase(j), fail);
        ok = __all_sync(kFull, ok);
        tc_fence_after();
        if (warp_ok && ok) {
          const int64_t left = s.t1 - s.t0 - int64_t(i) * TN;
          const int valid = int(left < TN ? left : TN);
          const uint32_t sb = tl + uint32_t(L::S + (j & 1) * TN);
          const uint32_t nk = L::NK + uint32_t(j & 3) * (TN * 4), nv = L::NV + uint32_t(j & 3) * (TN * 4);
          // the largest ν^K·S of the row
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < TN / 64; ++h) {
            uint32_t v[2][32];
            tmem_ld32(sb + 64 * h, v[0]);
            tmem_ld32(sb + 64 * h + 32, v[1]);
            tmem_ld_wait();
            auto fold = [&](auto full) {
#pragma unroll
              for (int k = 0; k < 64; k += 4) {
                const float4 n = lds_f4(nk + uint32_t(64 * h + k) * 4);
                const uint32_t* x = &v[k >> 5][k & 31];
                const float2 y0 = mul2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), make_float2(n.x, n.y));
                const float2 y1 = mul2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), make_float2(n.z, n.w));
                if constexpr (decltype(full)::value) {
                  mx = fmaxf(fmaxf(mx, fmaxf(y0.x, y0.y)), fmaxf(y1.x, y1.y));
                } else {
                  const int t = 64 * h + k;
                  if (t < valid) mx = fmaxf(mx, y0.x);
                  if (t + 1 < valid) mx = fmaxf(mx, y0.y);
                  if (t + 2 < valid) mx = fmaxf(mx, y1.x);
                  if (t + 3 < valid) mx = fmaxf(mx, y1.y);
                }
              }
            };
            if (valid == TN) fold(std::true_type{});
            else fold(std::false_type{});
          }
          mx *= rs;
          const float4 vm = lds_f4(L::VMAX + uint32_t(j & 3) * 16);
          const float big = TN == 128 ? fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w)) : fmaxf(vm.x, vm.y);
          const float pw = fminf(fmaxf(__uint_as_float(__float_as_uint(big) & 0x7f800000u), 0x1p-60f), 0x1p60f);
          if (i == 0) {
            m = mx;
            vn = pw;
            mp = m - 8.f + float(int(__float_as_uint(vn) >> 23) - 127);
          } else {
            const bool up = mx > m + 4.f, wide = pw > 4.f * vn;
            if (__any_sync(kFull, up || wide)) {
              if (up) m = mx;
              if (wide) vn = pw;
              const float mn = m - 8.f + float(int(__float_as_uint(vn) >> 23) - 127);
              const float f = ex2(mp - mn);
              mp = mn;
              l2 = mul2(l2, make_float2(f, f));
              ok = __all_sync(kFull, wait_for(o_done(j - 1), phase(j - 1), fail));
              tc_fence_after();
              if (ok) {
#pragma unroll 1
                for (int k = 0; k < D; k += 16) {
                  uint32_t o[16];
                  tmem_ld16(tl + uint32_t(L::O + k), o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st16(tl + uint32_t(L::O + k), o);
                }
                tmem_st_wait();
              }
            }
          }
          // weights into S's columns, the sum of the exponentials
          const float2 rs2 = make_float2(rs, rs), mp2 = make_float2(-mp, -mp);
#pragma unroll
          for (int h = 0; h < TN / 32; ++h) {
            uint32_t v[32], p[16];
            tmem_ld32(sb + 32 * h, v);
            tmem_ld_wait();
            auto weigh = [&](auto full) {
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 n = lds_f4(nk + uint32_t(32 * h + k) * 4), w = lds_f4(nv + uint32_t(32 * h + k) * 4);
                const float2 x0 = fma2(mul2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), make_float2(n.x, n.y)), rs2, mp2);
                const float2 x1 = fma2(mul2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), make_float2(n.z, n.w)), rs2, mp2);
                float2 e0 = make_float2(ex2(x0.x), ex2(x0.y)), e1 = make_float2(ex2(x1.x), ex2(x1.y));
                if constexpr (!decltype(full)::value) {
                  const int t = 32 * h + k;
                  if (t >= valid) e0.x = 0.f;
                  if (t + 1 >= valid) e0.y = 0.f;
                  if (t + 2 >= valid) e1.x = 0.f;
                  if (t + 3 >= valid) e1.y = 0.f;
                }
                l2 = add2(l2, e0);
                l2 = add2(l2, e1);
                const float2 w0 = mul2(e0, make_float2(w.x, w.y)), w1 = mul2(e1, make_float2(w.z, w.w));
                const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
                p[k / 2] = *reinterpret_cast<const uint32_t*>(&h0);
                p[k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
              }
            };
            if (valid == TN) weigh(std::true_type{});
            else weigh(std::false_type{});
            tmem_st16(sb + 16 * h, p);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(j));
      }
      // the segment's state
      ok = ok && wait_for(o_done(j - 1), phase(j - 1), fail);
      ok = __all_sync(kFull, ok);
      tc_fence_after();
      if (warp_ok) {
        const int64_t st = s.state + tid;
        if (row_ok)
          a.stats[st] = ok ? make_float2(mp, l2.x + l2.y) : make_float2(__uint_as_float(0x7fc00000u), 0.f);
        if (ok) {
#pragma unroll 1
          for (int k = 0; k < D; k += 32) {
            uint32_t o[32];
            tmem_ld32(tl + uint32_t(L::O + k), o);
            tmem_ld_wait();
            if (row_ok) {
              float* dst = a.acc + st * D + k;
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + e), "r"(o[e]), "r"(o[e + 1]),
                             "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]), "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                             : "memory");
            }
          }
        }
      }
      c.i = s.tiles - 1;
      c.next(a);
    }
  } else if (warp < kSoftWarps + kFillWarps) {
    // ------------------------------------------------------------ codes to fp16 levels in shared memory
    const int ft = tid - kSoftWarps * 32;
    const int tok = ft % TN, sub = ft / TN;               // K: one token, OCT octets from sub·OCT
    const int c0 = (sub * L::OCT) & 7, kblock = sub * L::OCT / 8;
    const int kb = lane & 7, rest = ft >> 3;              // V: 8 tokens, one octet
    const int vo = rest % (D / 8), vblock = rest / (D / 8);
    const bool v_mine = vblock < TN / 64;
    const uint32_t kword = L::TABLE | uint32_t(lane * 4), vword = kword | 128u;
    const uint32_t krow = uint32_t(kblock) * (TN * 128) + uint32_t(tok) * 128;
    const uint32_t vrow = uint32_t(vblock) * (D * 128) + uint32_t(8 * vo) * 128;
    uint32_t kw[8], vw[16];
    float norm_k = 0.f, norm_v = 0.f;
    auto fetch_k = [&](const Cursor& c) {
      const Segment& s = c.s;
      const int64_t t = s.t0 + int64_t(c.i) * TN + tok;
      const int64_t row = (s.token_base + (t < s.t1 ? t : s.t1 - 1)) * a.hkv + s.g;
      const uint8_t* base = a.k_codes[s.part] + row * (D * a.k_bits / 8) + sub * L::OCT * a.k_bits;
      switch (a.k_bits) {
        case 1: load_k<1, L::OCT>(base, kw); break;
        case 2: load_k<2, L::OCT>(base, kw); break;
        case 3: load_k<3, L::OCT>(base, kw); break;
        default: load_k<4, L::OCT>(base, kw); break;
      }
      if (sub == 0) {
        norm_k = __ldg(a.k_norms[s.part] + row);
        norm_v = t < s.t1 ? __ldg(a.v_norms[s.part] + row) : 0.f;
      }
    };
    auto fetch_v = [&](const Cursor& c) {
      if (!v_mine) return;
      const Segment& s = c.s;
      const uint8_t* p[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int64_t t = s.t0 + int64_t(c.i) * TN + 64 * vblock + 8 * kb + r;
        p[r] = a.v_codes[s.part] + ((s.token_base + (t < s.t1 ? t : s.t1 - 1)) * a.hkv + s.g) * (D * a.v_bits / 8);
      }
      switch (a.v_bits) {
        case 1: load_v<1>(p, vo, vw); break;
        case 2: load_v<2>(p, vo, vw); break;
        case 3: load_v<3>(p, vo, vw); break;
        default: load_v<4>(p, vo, vw); break;
      }
    };
    Cursor c(a, range);
    if (c.live()) {
      fetch_k(c);
      fetch_v(c);
    }
    bool ok = placed;
    for (int j = 0; c.live(); ++j) {
      Cursor n = c;
      n.next(a);
      if (j >= 2) ok = ok && wait_for(s_full(j), phase(j - 2), fail);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      if (sub == 0) {
        const uint32_t slot = uint32_t(j & 3) * (TN * 4) + uint32_t(tok) * 4;
        *reinterpret_cast<float*>(at(L::NK + slot)) = norm_k;
        *reinterpret_cast<float*>(at(L::NV + slot)) = norm_v;
        float big = norm_v;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
        if (lane == 0) *reinterpret_cast<float*>(at(L::VMAX + uint32_t(j & 3) * 16 + uint32_t(tok >> 5) * 4)) = big;
      }
      {
        const uint32_t row = (j & 1 ? L::K1 : L::K0) + krow;
        switch (a.k_bits) {
          case 1: put_k<1, L::OCT>(kw, row, c0, tok, kword); break;
          case 2: put_k<2, L::OCT>(kw, row, c0, tok, kword); break;
          case 3: put_k<3, L::OCT>(kw, row, c0, tok, kword); break;
          default: put_k<4, L::OCT>(kw, row, c0, tok, kword); break;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full(j));
      if (n.live()) fetch_k(n);
      if (j >= 2) ok = wait_for(o_done(j), phase(j - 2), fail);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      if (v_mine) {
        const uint32_t row = L::V0 + uint32_t(j & 1) * 0x8000u + vrow;
        switch (a.v_bits) {
          case 1: put_v<1>(vw, vo, row, kb, vword); break;
          case 2: put_v<2>(vw, vo, row, kb, vword); break;
          case 3: put_v<3>(vw, vo, row, kb, vword); break;
          default: put_v<4>(vw, vo, row, kb, vword); break;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(j));
      if (n.live()) fetch_v(n);
      c = n;
    }
  } else if (lane == 0) {
    // ---------------------------------------------------------------- one thread issues the products
    Cursor c(a, range);
    int j = 0, seg = 0;
    bool ok = placed;
    auto scores = [&](int jj) {
      const uint32_t d = tmem + uint32_t(L::S + (jj & 1) * TN), k = jj & 1 ? L::K1 : L::K0;
#pragma unroll
      for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_f16_ts(d, tmem + uint32_t((part ? L::QL : L::Q) + 8 * ks),
                        smem_desc_sw128(k + uint32_t(ks >> 2) * (TN * 128) + uint32_t(ks & 3) * 32), L::idesc(TN),
                        uint32_t(part + ks > 0));
      mma_commit(s_full(jj));
    };
    while (ok && c.live()) {
      const int tiles = c.s.tiles;
      ok = wait_for(q_full, uint32_t(seg) & 1u, fail) && wait_for(k_full(j), phase(j), fail);
      if (!ok) break;
      tc_fence_after();
      scores(j);
      for (int i = 0; i < tiles; ++i, ++j) {
        if (i + 1 < tiles) {
          ok = wait_for(k_full(j + 1), phase(j + 1), fail) && (j < 1 || wait_for(o_done(j - 1), phase(j - 1), fail));
          if (!ok) break;
          tc_fence_after();
          scores(j + 1);
        }
        ok = wait_for(v_full(j), phase(j), fail) && wait_for(p_full(j), phase(j), fail);
        if (!ok) break;
        tc_fence_after();
        const uint32_t p = tmem + uint32_t(L::S + (j & 1) * TN), v = L::V0 + uint32_t(j & 1) * 0x8000u;
#pragma unroll
        for (int ks = 0; ks < TN / 16; ++ks)
          tc_mma_f16_ts(tmem + uint32_t(L::O), p + uint32_t(8 * ks),
                        smem_desc_sw128(v + uint32_t(ks >> 2) * (D * 128) + uint32_t(ks & 3) * 32), L::idesc(D),
                        uint32_t(i > 0 || ks > 0));
        mma_commit(o_done(j));
      }
      ++seg;
      c.i = tiles - 1;
      c.next(a);
    }
    // products still in flight end before the tensor memory is given up
    uint64_t* drain = &bars[11];
    mbar_init(drain, 1);
    fence_mbarrier_init();
    mma_commit(drain);
    for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(drain, 0); ++i) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int D, bool SPLIT> cudaError_t launch_split(const SharedArgs& a, cudaStream_t stream) {
  auto k = shared_tc_kernel<D, SPLIT>;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(Tc<D>::kTotal));
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(unsigned(a.grid)), dim3(kThreads), Tc<D>::kTotal, stream, a);
}

}  // namespace

cudaError_t launch_shared_tc(const SharedArgs& a, cudaStream_t stream) {
  int dev = 0, reserved = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e != cudaSuccess) return e;
  if (uint32_t(reserved) != Tc<128>::kBase) return cudaErrorNotSupported;
  if (a.d == 64) return a.split ? launch_split<64, true>(a, stream) : launch_split<64, false>(a, stream);
  if (a.d == 128) return a.split ? launch_split<128, true>(a, stream) : launch_split<128, false>(a, stream);
  return launch_split<256, false>(a, stream);
}

}  // namespace rrq
