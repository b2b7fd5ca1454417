// attention_shared_tc.cu — partial states of attention over a quantised cache on the
// 5th-generation tensor cores, for head sizes up to 256: up to 128 query rows against a
// run of tiles of one kv head (attention_shared.h).
//
// With the rows' rotated queries q' (two fp16 parts, the second what the first rounds off, and a
// power of two 2^-e per row taken out) and the levels c as fp16,
//     S = Q'·C_Kᵀ,   x = 2^e·ν^K_t·S,   P = 2^{x − m'}·ν^V_t,   O += P·C_V,
// where m' = m − 9 follows the row's running maximum m of x + log2 ν^V (so of the products
// that are summed: a token with most of the weight and a value of no size does not push the
// others out of fp16's range, nor does a large value without weight).  It moves only when m
// grows by more than 6 (powers of two), so O is rarely rescaled; P is at most 2^15.  In a full
// tile whose value norms lie within 2^5 of one another max x + max log2 ν^V stands for the
// maximum, at most 5 above it, without a second number per token (64 sequences on a prefix of
// 32768 tokens: 125 us; 152 where the norms' logarithms deviate by 1, so that no tile is of
// that kind); so P keeps 11 bits down to 2^-18 of the row's largest at least.  It is one fp16
// part: 2^-12 of a weight on average, no more than fp16 outputs are rounded by, while a second
// would take another product.  Norms below 2^-90 count as 2^-90 in m, which keeps 2^{x − m'}
// and its sum within fp32's range.  The state (m', Σ 2^{x − m'}, O) is what the merge takes.
//
// Units of at most 16 rows (d ≤ 128) exchange the operands' roles: a tile's 128 tokens are the
// rows of Sᵀ = C_K·Q'ᵀ and the coordinates the rows of Oᵀ = C_Vᵀ·Pᵀ, 16 columns wide, so that a
// thread has a token's 8 rows to weigh instead of a row's 64 tokens of which most
// rows would be empty (33 sequences x 4 heads of up to 1500 tokens, 4 rows a unit: 22 us against 33
// without; 64 x 8 tails behind a prefix of 32768 tokens: 128 against 168).
//
// Bound by the latency of the weight warps' two passes (about 3600 of a tile's 4400 cycles at 128
// rows): 64 sequences x 32 heads on 32768 + 1024 tokens x 8 heads take 125 us, 280 TFLOP/s,
// against 21 us of products at the tensor cores' rate (32 with the queries' second part); 16
// sequences on 4096 tokens 28 us.
//
// One CTA per SM walks its range of tiles (128 tokens, 64 for d = 256), 19 warps:
//  * warp 17 copies the packed codes of two tiles ahead into shared memory (TMA boxes of
//    half a tile's rows, swizzled where rows are 32, 64 or 128 bytes; rows of 8 and 24 bytes
//    are not multiples of TMA's 16 and are read by the filling warps themselves);
//  * warps 8–11 and 12–15 turn K and V codes into fp16 levels, one token per thread, by one
//    shared-memory lookup per byte of two coordinates (tables of 256 pairs, one copy per lane
//    so that no bank conflicts; at d = 256 eight copies), and write rows [token][coordinate] in the 128-byte swizzle,
//    K in two stages: as they lie, K is a K-major operand and V, whose tokens are summed over,
//    an MN-major one.  Row 8k + e of a tile's 64 is token 8k + (e + k) mod 8, so the eight
//    lanes that share a wavefront read eight neighbouring code rows;
//  * warp 16 issues S, a tile ahead of the weights, and warp 18 O;
//  * warps 0–7 make the weights: two threads per query row with half of the tokens each,
//    the row's maximum met through shared memory, weights back into S's own columns as
//    fp16 (or, for few rows, a thread per token and 8 rows, weights into shared memory).
// Tensor memory: S twice, O and the queries, of which d = 256 has room for the first part only (512
// columns in use): its second part is an operand in shared memory, in place of three quarters of
// the tables' copies and of what few rows take elsewhere (32 sequences x 32/8 heads on 8192
// tokens 65 us, with one part of 11 bits and all copies 52; 7 x 16/4 heads on 2049: 25 and 22).
// Every wait is bounded; a wait that gives up makes the CTA's states NaN.
#include <cstring>

#include "attention_shared.cuh"
#include "cluster.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace rrq {
namespace {

constexpr uint32_t kWaitLimit = 1u << 24;  // polls, a few seconds in all
constexpr int kSoftWarps = 8, kFillWarps = 8;
constexpr int kFill = 128;  // threads that fill K, and as many that fill V
constexpr float kGrowth = 6.f, kRoom = 9.f;  // of a row's maximum before m' moves; of the weights above it
constexpr float kTight = 5.f;  // powers of two that a tile's value norms may span for the short way to m
// Rows of a unit that exchanges the operands' roles, as many as its 16 columns hold: 33 x 4 tails of up
// to 1500 tokens at 4, 8, 12 and 16 rows 22, 23, 24 and 24 us (30, 32, 36 and 36 without); one
// sequence of 65536 tokens x 8 heads 53, 54, 57 and 57 (63, 65, 65 and 66).
constexpr int kFewRows = 16;
constexpr int kThreads = (kSoftWarps + kFillWarps + 3) * 32;

template <int D> struct Tc {
  static constexpr int TN = D <= 128 ? 128 : 64;     // tokens per tile
  static constexpr int TURNS = D / 32 * TN / kFill;  // turns of 4 octets per filling thread (a token's, or half a token's)
  static constexpr int PR = TN / 2;                  // rows of a piece of packed codes
  static constexpr uint32_t TILE = TN * D * 2;       // bytes of a K or V stage
  // shared addresses (the dynamic base is checked to be kBase)
  static constexpr uint32_t kBase = 0x400;
  static constexpr uint32_t BARS = 0x400;
  static constexpr uint32_t TSLOT = 0x4C0;
  static constexpr uint32_t FAIL = 0x4D0;
  static constexpr uint32_t LRANGE = 0x600;          // [4 tiles][max, −min][4 warps] of the logarithms below
  static constexpr uint32_t NK = 0x800, NV = 0x1000, LV = 0x1800;  // [4 tiles][TN] norms, log2 of the value norms
  static constexpr uint32_t PT = 0x2000;             // few rows: weights [2 tiles][2 × 64 tokens][16 rows], swizzled
  static constexpr uint32_t QB = 0x4000;             // few rows: queries [part][64 coordinates][16 rows], swizzled
  static constexpr uint32_t RS = 0x580;              // few rows: [2 segments][16] powers of two taken out of the queries
  static constexpr uint32_t XCH = 0x6000;            // [2 tiles][2 halves][128 rows] maxima
  // packed codes: eight 4 KB pieces of half a tile's rows, at most 64 (d = 256: 128) bytes each
  __host__ __device__ static constexpr uint32_t piece(int stage, int v, int half) {
    return 0x8000u + uint32_t(stage * 4 + v * 2 + half) * 0x1000u;
  }
  // pairs of levels, COPIES to an entry: K and V alternating (32) or one table after the other (8)
  static constexpr int COPIES = D <= 128 ? 32 : 8;
  static constexpr uint32_t TABLE = 0x10000, VTABLE = COPIES == 32 ? COPIES * 4 : 256 * COPIES * 4;
  static constexpr uint32_t K0 = 0x20000;            // K stages of 32 KB
  // d = 256: second query part, 64 coordinates of the 128 rows per block of 16 KB, swizzled
  __host__ __device__ static constexpr uint32_t qlow(int block) { return block < 3 ? 0x14000u + uint32_t(block) * 0x4000u : 0x2000u; }
  static constexpr uint32_t VT = 0x30000;            // V tile
  static constexpr size_t kTotal = 0x38000 - kBase;
  // tensor memory columns
  static constexpr int S = 0, O = 2 * TN, Q = O + D, QL = Q + D / 2;
  // fp16 operands, fp32 sums, M = 128; bits 15 and 16: A, B MN-major
  static constexpr uint32_t idesc(int n) { return (1u << 4) | (uint32_t(n / 8) << 17) | ((128u / 16) << 24); }
  static_assert(LV + 4 * TN * 4 <= PT && TABLE + 256 * 2 * COPIES * 4 <= (D <= 128 ? K0 : 0x14000u) && TILE <= 0x8000 &&
                    kTotal <= 227 * 1024, "layout");
};

// Token of row (column of S) n of a tile.
__host__ __device__ constexpr int token_of(int n) { return (n & ~7) | ((n + (n >> 3)) & 7); }

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* fail) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *fail) return false;
  }
  *fail = 1;
  return false;
}
// True in one thread of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle: rows of 64 MN
// elements, one per K index, eight rows to a 1024-byte group; `block`: bytes from one run
// of 64 MN elements to the next.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= uint64_t((saddr >> 4) & 0x3FFFu);
  d |= uint64_t((block >> 4) & 0x3FFFu) << 16;  // leading offset: along MN
  d |= uint64_t(1024u >> 4) << 32;              // stride offset: along K
  d |= uint64_t(1) << 46;                       // descriptor version for sm_100
  d |= uint64_t(2) << 61;                       // layout: 128-byte swizzle
  return d;
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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
// AND of `v` over the `nthreads` threads (whole warps) meeting at named barrier `id`.
__device__ __forceinline__ bool meet(uint32_t id, uint32_t nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(v)), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// log2 of a value norm for the running maximum; the approximation's error (2^-22) only moves m.
__device__ __forceinline__ float norm_log2(float norm) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(fabsf(norm), 0x1p-90f)));
  return y;
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

struct SharedMaps {
  CUtensorMap k[2], v[2];  // prefix, tails
};

// Rows that TMA can move; the others are read from global memory by the filling warps.
template <int D, int B> constexpr bool kBoxed = D * B / 8 % 16 == 0;

// Byte `off` of row r in a piece of packed codes (the swizzle of head_rows_tensor_map).
template <int PITCH> __device__ __forceinline__ uint32_t code_at(int r, uint32_t off) {
  const uint32_t x = PITCH == 128 ? uint32_t(r) & 7u : PITCH == 64 ? uint32_t(r >> 1) & 3u : PITCH == 32 ? uint32_t(r >> 2) & 1u : 0u;
  return uint32_t(r) * PITCH + (off ^ (x << 4));
}
__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
// A shared word that is written again later (lds_u32 is for constant tables).
__device__ __forceinline__ uint32_t lds_word(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// ---- the filling warps' reads, by code width
// Four octets (B words) of a code row, number `it`, from a piece (row r).
template <int D, int B> __device__ __forceinline__ void read_octets(uint32_t piece, int r, int it, uint32_t (&w)[4]) {
  constexpr int PITCH = D * B / 8;
  const uint32_t off = uint32_t(it) * (4 * B);
  if constexpr (B == 4) {
    const uint4 v = lds_u4(piece + code_at<PITCH>(r, off));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (B == 2) {
    const uint2 v = lds_u2(piece + code_at<PITCH>(r, off));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = lds_word(piece + code_at<PITCH>(r, off + 4 * i));
  }
}
// Octet i of four, as nibbles.
template <int B> __device__ __forceinline__ uint32_t octet_of(const uint32_t (&w)[4], int i) {
  if constexpr (B == 4) return w[i];
  const int bit = 8 * B * i, k = bit >> 5, sh = bit & 31;
  uint32_t v = w[k] >> sh;
  if (sh + 8 * B > 32) v = __funnelshift_r(w[k], w[k + 1 < 4 ? k + 1 : 3], sh);
  return octet_nibbles(v & (B == 3 ? 0xffffffu : B == 2 ? 0xffffu : 0xffu), B);
}
// The largest and the smallest logarithm of a tile's value norms, as the K-filling warps left them.
template <int TN> __device__ __forceinline__ float2 log2_range(uint32_t at, int j) {
  const float4 a = lds_f4(at + uint32_t(j & 3) * 32), b = lds_f4(at + uint32_t(j & 3) * 32 + 16);
  float2 r = make_float2(fmaxf(a.x, a.y), fmaxf(b.x, b.y));
  if (TN == 128) r = make_float2(fmaxf(r.x, fmaxf(a.z, a.w)), fmaxf(r.y, fmaxf(b.z, b.w)));
  return make_float2(r.x, -r.y);
}
// Level pair of byte k of `w`; `lane_word` = table | copy of the lane.  Entries of 256 or 32 bytes.
template <int COPIES, int K> __device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t lane_word) {
  if constexpr (COPIES == 32)
    return lds_u32(__byte_perm(w, lane_word, K == 0 ? 0x7604u : K == 1 ? 0x7614u : K == 2 ? 0x7624u : 0x7634u));
  else
    return lds_u32(((K == 0 ? w << 5 : w >> (8 * K - 5)) & 0x1fe0u) | lane_word);
}

// Four octets of a token's row as levels, chunks c0 .. c0 + 3 of `row`.  All
// lookups come before the first store: a load is not moved ahead of a store that might alias it.
template <int COPIES, int B> __device__ __forceinline__ void put_octets(const uint32_t (&w)[4], uint32_t row, int c0, int n, uint32_t lane_word) {
  uint32_t p[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = octet_of<B>(w, i);
    p[i][0] = pair_of<COPIES, 0>(x, lane_word), p[i][1] = pair_of<COPIES, 1>(x, lane_word);
    p[i][2] = pair_of<COPIES, 2>(x, lane_word), p[i][3] = pair_of<COPIES, 3>(x, lane_word);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    sts_v4(row + (uint32_t((c0 + i) ^ (n & 7)) << 4), p[i][0], p[i][1], p[i][2], p[i][3]);
}

// Columns [h, h + 32) of a tile: `v` where the column's token is not one of the first `valid`.
__device__ __forceinline__ void mask(float2 (&y)[16], int h, int valid, float v) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int n = h + 2 * k;
    if (token_of(n) >= valid) y[k].x = v;
    if (token_of(n + 1) >= valid) y[k].y = v;
  }
}

// The largest x + log2 ν over columns [from, from + TN/2) of a tile, token by token (`sb`: their tensor
// memory, `nk`: their key norms).  Not inlined: next to the common way it cost registers there, 133 us
// instead of 125 for 64 sequences on a prefix of 32768 tokens.
template <int TN, bool WHOLE> __device__ __noinline__ float largest_sum(uint32_t sb, uint32_t nk, int from, int valid, float rs) {
  const uint32_t lv = nk + (Tc<128>::LV - Tc<128>::NK);  // for every D
  const float2 rs2 = make_float2(rs, rs);
  float mx = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < TN / 2; h += 32) {
    uint32_t v[32];
    tmem_ld32(sb + h, v);
    tmem_ld_wait();
    float2 y[16];
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 n = lds_f4(nk + uint32_t(h + k) * 4), g = lds_f4(lv + uint32_t(h + k) * 4);
      const float2 s0 = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
      const float2 s1 = make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
      y[k / 2] = fma2(mul2(s0, make_float2(n.x, n.y)), rs2, make_float2(g.x, g.y));
      y[k / 2 + 1] = fma2(mul2(s1, make_float2(n.z, n.w)), rs2, make_float2(g.z, g.w));
    }
    if constexpr (!WHOLE) mask(y, from + h, valid, -INFINITY);
#pragma unroll
    for (int k = 0; k < 16; k += 2) mx = fmaxf(mx, fmaxf(fmaxf(y[k].x, y[k].y), fmaxf(y[k + 1].x, y[k + 1].y)));
  }
  return mx;
}

// Position in a range's segments, one tile at a time.
struct Cursor {
  int index, i;  // the segment (−1 at the end), the tile in it
  SharedSegment s;
  __device__ __forceinline__ Cursor(const SharedArgs& a, int range) : index(a.begin[range]), i(0) {
    if (index >= 0) load(a);
  }
  __device__ __forceinline__ void load(const SharedArgs& a) {
    s = shared_segment(a, index);
    if (!(s.flags & 2)) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.segs + 2 * (index + 1)));
  }
  __device__ __forceinline__ bool live() const { return index >= 0; }
  __device__ __forceinline__ void next_segment(const SharedArgs& a) {
    i = 0;
    index = s.flags & 2 ? -1 : index + 1;
    if (index >= 0) load(a);
  }
  __device__ __forceinline__ void next(const SharedArgs& a) {
    if (++i == s.tiles) next_segment(a);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ SharedMaps maps) {
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
  auto c_full = [&](int j, bool v) { return &bars[(v ? 17 : 12) + (j & 1)]; };
  auto c_free = [&](int j, bool v) { return &bars[(v ? 19 : 14) + (j & 1)]; };
  auto phase = [](int j) { return uint32_t(j >> 1) & 1u; };
  uint32_t* tslot = reinterpret_cast<uint32_t*>(at(L::TSLOT));
  volatile int* fail = reinterpret_cast<volatile int*>(at(L::FAIL));
  const bool placed = smem_addr(dsm) == L::kBase;  // the launch checks it too

  if (tid == 0) {
    mbar_init(q_full, kSoftWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), kFillWarps / 2);
      mbar_init(v_full(s), kFillWarps / 2);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), kSoftWarps);
      mbar_init(o_done(s), 1);
      for (int v = 0; v < 2; ++v) {
        mbar_init(c_full(s, v), 1);
        mbar_init(c_free(s, v), kFillWarps / 2);
      }
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
  for (int i = tid; i < 256 * 2 * L::COPIES && placed; i += kThreads) {
    const int v = (i / L::COPIES) & 1, b = i / (2 * L::COPIES);
    const float* lev = v ? a.v_levels : a.k_levels;
    const float f = v ? a.v_alpha : a.k_alpha;
    const __half2 h = __floats2half2_rn(lev[b & 15] * f, lev[b >> 4] * f);
    const uint32_t entry = L::COPIES == 32 ? uint32_t(b) * 256 : uint32_t(b) * (L::COPIES * 4);
    *reinterpret_cast<__half2*>(at(L::TABLE + entry + (v ? L::VTABLE : 0u) + uint32_t(i & (L::COPIES - 1)) * 4)) = h;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();  // from here on, global memory

  if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- weights
    const int quarter = warp & 3, half = warp >> 2;  // tensor-memory lanes, half of the tokens (of the rows)
    const int ln = 32 * quarter + lane;              // this thread's tensor-memory lane
    const uint32_t tl = tmem + (uint32_t(32 * quarter) << 16);
    Cursor c(a, range);
    int j = 0, seg = 0;
    bool staged = false;  // the segment's queries are in shared memory already
    // few rows: the queries of a segment as an operand, rows past its own as zeros; read from
    // global memory a segment before they are staged
    uint4 qv[2];
    float qe = 1.f;
    const int q_row = (tid >> 3) & 15, q_chunk = (tid & 7) + ((tid >> 7) << 3);  // row, chunk of 8 coordinates
    auto read_queries = [&](const SharedSegment& s) {
      const int64_t qrow = int64_t(s.g) * a.rows + s.row0;
      if (q_row < s.nrows && q_chunk < D / 8) {
#pragma unroll
        for (int part = 0; part < 2; ++part)
          qv[part] = __ldcg(reinterpret_cast<const uint4*>((part ? a.ql : a.qh) + (qrow + q_row) * D) + q_chunk);
      }
      if (tid < 16 && tid < s.nrows) qe = __ldcg(a.qexp + qrow + tid);
    };
    auto stage = [&](const SharedSegment& s, int number) {
      if (q_chunk < D / 8) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint4 v = q_row < s.nrows ? qv[part] : make_uint4(0, 0, 0, 0);
          sts_v4(L::QB + uint32_t(part * (D / 64) + (q_chunk >> 3)) * 2048 + uint32_t(q_row) * 128 +
                     (uint32_t((q_chunk ^ q_row) & 7) << 4), v.x, v.y, v.z, v.w);
        }
      }
      if (tid < 16) *reinterpret_cast<float*>(at(L::RS + uint32_t(number & 1) * 64 + uint32_t(tid) * 4)) = tid < s.nrows ? qe : 1.f;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    while (c.live()) {
      const SharedSegment s = c.s;
      bool ok = *fail == 0;
      if (D <= 128 && s.nrows <= kFewRows) {
        if constexpr (D <= 128) {
          // ---- few rows: lane = token, columns = rows; this half's rows [8·half, + 8)
          const bool mine = 8 * half < s.nrows;
          if (!staged) {
            read_queries(s);
            stage(s, seg);
          }
          staged = false;
          if (!(s.flags & 2)) read_queries(shared_segment(a, c.index + 1));
          float rs[8], m[8], mp[8], l[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) m[r] = mp[r] = l[r] = 0.f;
          for (int i = 0; i < s.tiles; ++i, ++j) {
            ok = ok && wait_for(s_full(j), phase(j), fail);
            ok = __all_sync(kFull, ok);
            tc_fence_after();
            if (mine) {
              const bool live = token_of(ln) < s.tokens - i * TN;
              const uint32_t wm = L::XCH + uint32_t(j & 1) * 1024 + uint32_t(half) * 128;
              float y[8], nv = 0.f;
              if (ok) {
                uint32_t v[8];
                tmem_ld8(tl + uint32_t(L::S + (j & 1) * TN + 8 * half), v);
                const float nk = __uint_as_float(lds_word(L::NK + uint32_t(j & 3) * (TN * 4) + uint32_t(ln) * 4));
                nv = __uint_as_float(lds_word(L::NV + uint32_t(j & 3) * (TN * 4) + uint32_t(ln) * 4));
                const float lv = __uint_as_float(lds_word(L::LV + uint32_t(j & 3) * (TN * 4) + uint32_t(ln) * 4));
                tmem_ld_wait();
                if (i == 0) {
                  const float4 r0 = lds_f4(L::RS + uint32_t(seg & 1) * 64 + uint32_t(half) * 32);
                  const float4 r1 = lds_f4(L::RS + uint32_t(seg & 1) * 64 + uint32_t(half) * 32 + 16);
                  rs[0] = r0.x, rs[1] = r0.y, rs[2] = r0.z, rs[3] = r0.w, rs[4] = r1.x, rs[5] = r1.y, rs[6] = r1.z, rs[7] = r1.w;
                }
                float mx[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                  y[r] = __uint_as_float(v[r]) * nk;
                  mx[r] = warp_max(live ? fmaf(y[r], rs[r], lv) : -INFINITY);
                }
                if (lane < 2)
                  sts_v4(wm + uint32_t(quarter) * 32 + uint32_t(lane) * 16, __float_as_uint(lane ? mx[4] : mx[0]),
                         __float_as_uint(lane ? mx[5] : mx[1]), __float_as_uint(lane ? mx[6] : mx[2]),
                         __float_as_uint(lane ? mx[7] : mx[3]));
              }
              ok = meet(uint32_t(5 + half), 128, ok);
              if (ok) {
                float mx[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float4 x0 = lds_f4(wm + uint32_t(q) * 32), x1 = lds_f4(wm + uint32_t(q) * 32 + 16);
                  const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                  for (int r = 0; r < 8; ++r) mx[r] = q ? fmaxf(mx[r], x[r]) : x[r];
                }
                if (i == 0) {
#pragma unroll
                  for (int r = 0; r < 8; ++r) {
                    m[r] = mx[r];
                    mp[r] = m[r] - kRoom;
                  }
                } else {
                  bool up = false;
#pragma unroll
                  for (int r = 0; r < 8; ++r) up = up || mx[r] > m[r] + kGrowth;
                  if (up) {  // the same in every thread of the half
                    ok = __all_sync(kFull, wait_for(o_done(j - 1), phase(j - 1), fail));
                    tc_fence_after();
                    uint32_t o[8];
                    tmem_ld8(tl + uint32_t(L::O + 8 * half), o);
                    tmem_ld_wait();
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                      if (mx[r] > m[r] + kGrowth) m[r] = mx[r];
                      const float mn = m[r] - kRoom, f = ex2(mp[r] - mn);
                      mp[r] = mn;
                      l[r] *= f;
                      o[r] = __float_as_uint(__uint_as_float(o[r]) * f);
                    }
                    tmem_st8(tl + uint32_t(L::O + 8 * half), o);
                    tmem_st_wait();
                  }
                }
                const uint32_t pt = L::PT + uint32_t(j & 1) * 4096 + uint32_t(ln >> 6) * 2048 + uint32_t(ln & 7) * 2;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                  const float p = live ? ex2(fmaf(y[r], rs[r], -mp[r])) : 0.f;
                  l[r] += p;
                  const __half w = __float2half_rn(p * nv);
                  asm volatile("st.shared.b16 [%0], %1;" ::"r"(pt + uint32_t(8 * half + r) * 128 + (uint32_t(((ln >> 3) ^ r) & 7) << 4)),
                               "h"(*reinterpret_cast<const unsigned short*>(&w))
                               : "memory");
                }
                fence_proxy_async_smem();
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(j));
          }
          // the next segment's queries go in while this one's last product runs: S of all its
          // tiles is done
          c.next_segment(a);
          if (c.live() && c.s.nrows <= kFewRows) {
            stage(c.s, seg + 1);
            staged = true;
          }
          ok = ok && wait_for(o_done(j - 1), phase(j - 1), fail);
          ok = __all_sync(kFull, ok);
          tc_fence_after();
          if (mine) {
            // the half's sums over its tokens, four warps through shared memory
            const uint32_t wl = L::XCH + uint32_t(j & 1) * 1024 + uint32_t(half) * 128;
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(kFull, l[r], o);
            if (lane == 0) {
              sts_v4(wl + uint32_t(quarter) * 32, __float_as_uint(l[0]), __float_as_uint(l[1]), __float_as_uint(l[2]), __float_as_uint(l[3]));
              sts_v4(wl + uint32_t(quarter) * 32 + 16, __float_as_uint(l[4]), __float_as_uint(l[5]), __float_as_uint(l[6]), __float_as_uint(l[7]));
            }
            ok = meet(uint32_t(5 + half), 128, ok);
            if (quarter == 0 && lane < 8 && 8 * half + lane < s.nrows) {
              float sum = 0.f, mine_mp = mp[0];
#pragma unroll
              for (int q = 0; q < 4; ++q) sum += __uint_as_float(lds_word(wl + uint32_t(q) * 32 + uint32_t(lane) * 4));
#pragma unroll
              for (int r = 1; r < 8; ++r)
                if (lane == r) mine_mp = mp[r];
              a.stats[int64_t(s.state) * a.rows + s.row0 + 8 * half + lane] = ok ? make_float2(mine_mp, sum) : make_float2(__uint_as_float(0x7fc00000u), 0.f);
            }
            if (ok) {
              uint32_t o[8];
              tmem_ld8(tl + uint32_t(L::O + 8 * half), o);
              tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < 8; ++r)
                if (8 * half + r < s.nrows && ln < D)
                  a.acc[(int64_t(s.state) * a.rows + s.row0 + 8 * half + r) * D + ln] = __uint_as_float(o[r]);
            }
            // the next segment writes this slot of the exchange again
            meet(uint32_t(5 + half), 128, true);
          }
        }
      } else {
        // ---- lane = query row; this half's tokens [half·TN/2, + TN/2)
        constexpr int TH = TN / 2, DH = D / 2;
        const bool row_ok = ln < s.nrows, warp_ok = 32 * quarter < s.nrows;
        const int64_t qrow = int64_t(s.g) * a.rows + s.row0 + (row_ok ? ln : 0);
        float rs = 1.f;
        if (warp_ok) {
          rs = a.qexp[qrow];
          const uint4* qh = reinterpret_cast<const uint4*>(a.qh + qrow * D + half * DH);
          const uint4* ql = reinterpret_cast<const uint4*>(a.ql + qrow * D + half * DH);
#pragma unroll
          for (int part = 0; part < (D <= 128 ? 2 : 1); ++part) {
#pragma unroll 1
            for (int i = 0; i < DH / 32; ++i) {
              uint32_t r[16];
              uint4 low[D <= 128 ? 1 : 4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 v = __ldcg((part ? ql : qh) + 4 * i + k);
                r[4 * k] = v.x, r[4 * k + 1] = v.y, r[4 * k + 2] = v.z, r[4 * k + 3] = v.w;
                if constexpr (D > 128) low[k] = __ldcg(ql + 4 * i + k);
              }
              tmem_st16(tl + uint32_t((part ? L::QL : L::Q) + half * (DH / 2) + 16 * i), r);
              if constexpr (D > 128) {
#pragma unroll
                for (int k = 0; k < 4; ++k)  // chunk 4i + k of this half's coordinates
                  sts_v4(L::qlow(half * (DH / 64) + (i >> 1)) + uint32_t(ln) * 128 + (uint32_t((4 * i + k) ^ ln) & 7) * 16, low[k].x,
                         low[k].y, low[k].z, low[k].w);
              }
            }
          }
          tmem_st_wait();
          if constexpr (D > 128) fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);

        float m = 0.f, mp = 0.f;  // running maximum, m'
        float l = 0.f;
        const uint32_t pair = uint32_t(1 + quarter);
        for (int i = 0; i < s.tiles; ++i, ++j) {
          ok = ok && wait_for(s_full(j), phase(j), fail);
          ok = __all_sync(kFull, ok);
          tc_fence_after();
          if (warp_ok) {
            const int left = s.tokens - i * TN, valid = left < TN ? left : TN;
            const bool full = valid == TN;
            const uint32_t sb = tl + uint32_t(L::S + (j & 1) * TN + half * TH);
            const uint32_t nk = L::NK + uint32_t((j & 3) * TN + half * TH) * 4, nv = nk + (L::NV - L::NK);
            const uint32_t xch = L::XCH + uint32_t(j & 1) * 1024 + uint32_t(ln) * 4;
            const float2 rs2 = make_float2(rs, rs);
            float mx = -INFINITY;
            if (ok) {
              // the largest x + log2 ν of the row's half, by way of the largest x where the norms allow it
              // (loops kept rolled: unrolled, the warps' different code ran out of the instruction cache)
              const float2 range = log2_range<TN>(L::LRANGE, j);
              if (full && range.x - range.y <= kTight) {
#pragma unroll 1
                for (int h = 0; h < TH; h += 32) {
                  uint32_t v[32];
                  tmem_ld32(sb + h, v);
                  tmem_ld_wait();
                  float2 y[16];
#pragma unroll
                  for (int k = 0; k < 32; k += 4) {
                    y[k / 2] = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                    y[k / 2 + 1] = make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
                    const float4 n = lds_f4(nk + uint32_t(h + k) * 4);
                    y[k / 2] = mul2(y[k / 2], make_float2(n.x, n.y));
                    y[k / 2 + 1] = mul2(y[k / 2 + 1], make_float2(n.z, n.w));
                  }
#pragma unroll
                  for (int k = 0; k < 16; k += 2) mx = fmaxf(mx, fmaxf(fmaxf(y[k].x, y[k].y), fmaxf(y[k + 1].x, y[k + 1].y)));
                }
                mx = fmaf(mx, rs, range.x);
              } else {
                mx = full ? largest_sum<TN, true>(sb, nk, half * TH, valid, rs) : largest_sum<TN, false>(sb, nk, half * TH, valid, rs);
              }
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(xch + uint32_t(half) * 512), "f"(mx) : "memory");
            }
            ok = meet(pair, 64, ok);
            if (ok) {
              mx = fmaxf(mx, __uint_as_float(lds_word(xch + uint32_t(half ^ 1) * 512)));
              if (i == 0) {
                m = mx;
                mp = m - kRoom;
              } else {
                const bool up = mx > m + kGrowth;
                if (__any_sync(kFull, up)) {
                  if (up) m = mx;
                  const float mn = m - kRoom, f = ex2(mp - mn);
                  mp = mn;
                  l *= f;
                  ok = __all_sync(kFull, wait_for(o_done(j - 1), phase(j - 1), fail));
                  tc_fence_after();
#pragma unroll 1
                  for (int k = 0; k < DH; k += 32) {
                    uint32_t o[32];
                    tmem_ld32(tl + uint32_t(L::O + half * DH + k), o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st32(tl + uint32_t(L::O + half * DH + k), o);
                  }
                  tmem_st_wait();
                }
              }
              // weights into S's columns, the sum of the exponentials
              const float2 mp2 = make_float2(-mp, -mp);
              const uint32_t pb = sb;  // the first half of the columns that this thread reads
              float2 s2 = make_float2(0.f, 0.f), s3 = s2;
              auto weigh = [&](auto whole) {
#pragma unroll 1
                for (int h = 0; h < TH; h += 32) {
                  uint32_t v[32], p[16];
                  tmem_ld32(sb + h, v);
                  tmem_ld_wait();
                  float2 e[16];
#pragma unroll
                  for (int k = 0; k < 32; k += 4) {
                    float2 x0 = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                    float2 x1 = make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
                    const float4 n = lds_f4(nk + uint32_t(h + k) * 4);
                    x0 = mul2(x0, make_float2(n.x, n.y));
                    x1 = mul2(x1, make_float2(n.z, n.w));
                    x0 = fma2(x0, rs2, mp2);
                    x1 = fma2(x1, rs2, mp2);
                    e[k / 2] = make_float2(ex2(x0.x), ex2(x0.y));
                    e[k / 2 + 1] = make_float2(ex2(x1.x), ex2(x1.y));
                  }
                  if constexpr (!decltype(whole)::value) mask(e, half * TH + h, valid, 0.f);
#pragma unroll
                  for (int k = 0; k < 32; k += 4) {
                    float2 w0 = e[k / 2], w1 = e[k / 2 + 1];
                    s2 = add2(s2, w0);
                    s3 = add2(s3, w1);
                    const float4 w = lds_f4(nv + uint32_t(h + k) * 4);
                    w0 = mul2(w0, make_float2(w.x, w.y));
                    w1 = mul2(w1, make_float2(w.z, w.w));
                    const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
                    p[k / 2] = *reinterpret_cast<const uint32_t*>(&h0);
                    p[k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                  }
                  tmem_st16(pb + h / 2, p);
                }
              };
              if (full) weigh(std::true_type{});
              else weigh(std::false_type{});
              l += (s2.x + s2.y) + (s3.x + s3.y);
              tmem_st_wait();
            }
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
          const uint32_t xch = L::XCH + uint32_t(j & 1) * 1024 + uint32_t(ln) * 4;
          if (half) asm volatile("st.shared.f32 [%0], %1;" ::"r"(xch), "f"(l) : "memory");
          ok = meet(pair, 64, ok);
          const int64_t st = int64_t(s.state) * a.rows + s.row0 + ln;
          if (!half && row_ok)
            a.stats[st] = ok ? make_float2(mp, l + __uint_as_float(lds_word(xch))) : make_float2(__uint_as_float(0x7fc00000u), 0.f);
          if (ok) {
#pragma unroll 1
            for (int k = 0; k < DH; k += 32) {
              uint32_t o[32];
              tmem_ld32(tl + uint32_t(L::O + half * DH + k), o);
              tmem_ld_wait();
              if (row_ok) {
                float* dst = a.acc + st * D + half * DH + k;
#pragma unroll
                for (int e = 0; e < 32; e += 8)
                  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + e), "r"(o[e]), "r"(o[e + 1]),
                               "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]), "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                               : "memory");
              }
            }
          }
          meet(pair, 64, true);  // the next segment writes this slot of the exchange again
        }
        c.next_segment(a);
      }
      ++seg;
    }
  } else if (warp < kSoftWarps + kFillWarps) {
    // ------------------------------------------------------------ codes to fp16 levels in shared memory
    // Four warps for K, four for V, the same code; the K side also leaves the norms for the weights.
    const bool v_side = warp >= kSoftWarps + kFillWarps / 2;
    const int ft = (tid - kSoftWarps * 32) & (kFill - 1);
    const int n = ft % TN, sub = ft / TN;  // row of the tile
    const int tok = token_of(n);
    const int bits = v_side ? a.v_bits : a.k_bits;
    const uint32_t lane_word = L::TABLE | uint32_t((lane & (L::COPIES - 1)) * 4) | (v_side ? L::VTABLE : 0u);
    const uint32_t piece0 = L::piece(0, v_side, tok / L::PR);
    Cursor c(a, range);
    uint32_t kw[2][4];  // rows that no box moves (d = 64)
    float norm_k = 0.f, norm_v = 0.f;
    // what comes from global memory for the cursor's tile, past L1 as it is read once; rows past the
    // end repeat the last
    auto fetch = [&] {
      const int tt = c.i * TN + tok, part = c.s.flags & 1;
      const bool in = tt < c.s.tokens;
      const int64_t row = int64_t(c.s.token + (in ? tt : c.s.tokens - 1)) * a.hkv + c.s.g;
      if (!v_side) {
        norm_k = __ldcg(a.k_norms[part] + row);
        norm_v = in ? __ldcg(a.v_norms[part] + row) : 0.f;
      }
      if constexpr (D == 64) {
        if (bits & 1) {
          const uint32_t* p = reinterpret_cast<const uint32_t*>((v_side ? a.v_codes : a.k_codes)[part] + row * (D * bits / 8));
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 3; ++k)
              if (k < bits) kw[i][k] = __ldcg(p + i * bits + k);
        }
      }
    };
    if (c.live()) fetch();
    bool ok = placed;
    for (int j = 0; c.live(); ++j) {
      // the codes are there; K's stage has been read by S of the last tile but one, V's tile by
      // O of the last
      ok = ok && wait_for(c_full(j, v_side), phase(j), fail);
      if (v_side) ok = ok && (j < 1 || wait_for(o_done(j - 1), phase(j - 1), fail));
      else ok = ok && (j < 2 || wait_for(s_full(j), phase(j - 2), fail));
      if (!v_side && sub == 0) {
        // norm slots are used every fourth tile: what read this one before was done when S of
        // tile j − 2 began
        const uint32_t slot = uint32_t(j & 3) * (TN * 4) + uint32_t(n) * 4;
        *reinterpret_cast<float*>(at(L::NK + slot)) = norm_k;
        *reinterpret_cast<float*>(at(L::NV + slot)) = norm_v;
        const float lv = norm_log2(norm_v), hi = warp_max(lv), lo = warp_max(-lv);
        *reinterpret_cast<float*>(at(L::LV + slot)) = lv;
        if (lane < 2)
          *reinterpret_cast<float*>(at(L::LRANGE + uint32_t(j & 3) * 32 + uint32_t(lane) * 16 + uint32_t(n >> 5) * 4)) = lane ? lo : hi;
      }
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      const uint32_t dst = (v_side ? L::VT : L::K0 + uint32_t(j & 1) * 0x8000u) + uint32_t(n) * 128;
      const uint32_t piece = piece0 + uint32_t(j & 1) * 0x4000u;
      uint32_t cw[2][4];
      if constexpr (D == 64) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 3; ++k) cw[i][k] = kw[i][k];
      }
      // the next tile's norms are on their way while this one is filled
      c.next(a);
      if (c.live()) fetch();
      auto fill = [&](auto width) {
        constexpr int B = decltype(width)::value;
        if constexpr (kBoxed<D, B>) {
#pragma unroll 1
          for (int it = sub * L::TURNS; it < (sub + 1) * L::TURNS; ++it) {
            uint32_t w[4];
            read_octets<D, B>(piece, tok % L::PR, it, w);
            put_octets<L::COPIES, B>(w, dst + uint32_t(it >> 1) * (TN * 128), (it & 1) * 4, n, lane_word);
          }
        } else {
          put_octets<L::COPIES, B>(cw[0], dst, 0, n, lane_word);
          put_octets<L::COPIES, B>(cw[1], dst, 4, n, lane_word);
        }
      };
      switch (bits) {
        case 1: fill(std::integral_constant<int, 1>{}); break;
        case 2: fill(std::integral_constant<int, 2>{}); break;
        case 3: fill(std::integral_constant<int, 3>{}); break;
        default: fill(std::integral_constant<int, 4>{}); break;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(v_side ? v_full(j) : k_full(j));
        mbar_arrive(c_free(j, v_side));
      }
    }
  } else if (warp == kSoftWarps + kFillWarps + 1) {
    // ---------------------------------------------------------------- one thread copies the packed codes
    if (lane == 0) {
      const bool kbox = D * a.k_bits / 8 % 16 == 0, vbox = D * a.v_bits / 8 % 16 == 0;
      const int krow = D * a.k_bits / 8, vrow = D * a.v_bits / 8;
      // K a tile ahead of V, as the filling warps take them
      Cursor ck(a, range), cv = ck;
      int jk = 0, jv = 0;
      auto copy = [&](Cursor& c, int& j, bool v) {
        const int row = v ? vrow : krow;
        const bool box = v ? vbox : kbox;
        if (j >= 2 && !wait_for(c_free(j, v), phase(j - 2), fail)) return false;
        const uint32_t bar = smem_addr(c_full(j, v));
        mbarrier_expect_tx(bar, box ? uint32_t(TN * row) : 0u);
        const CUtensorMap* map = (v ? maps.v : maps.k) + (c.s.flags & 1);
        if (box) {
#pragma unroll
          for (int h = 0; h < 2; ++h)  // rows past the cache's end are filled with zeros
            tma_load_2d(L::piece(j & 1, v, h), map, c.s.g * row, c.s.token + c.i * TN + h * L::PR, bar);
        }
        c.next(a);
        ++j;
        return true;
      };
      bool ok = placed;
      while (ok && cv.live()) {
        if (ck.live()) ok = copy(ck, jk, false);
        if (ok && (jv + 1 < jk || !ck.live())) ok = copy(cv, jv, true);
      }
      // copies still in flight end before the CTA does
      for (int v = 0; v < 2; ++v) {
        const int n = v ? jv : jk;
        for (int k = n > 2 ? n - 2 : 0; k < n; ++k)
          for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(c_full(k, v), phase(k)); ++i) {
          }
      }
    }
  } else {
    // ---------------------------------------------------------------- products; the warps stay together, one thread issues
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    const bool o_side = warp == kSoftWarps + kFillWarps + 2;
    Cursor c(a, range);
    int j = 0, seg = 0;
    bool ok = placed;
    for (; ok && c.live(); c.next_segment(a), ++seg) {
      const int tiles = c.s.tiles;
      const bool few = D <= 128 && c.s.nrows <= kFewRows;
      if (!o_side) {
        ok = __all_sync(kFull, wait_for(q_full, uint32_t(seg) & 1u, fail));
        for (int i = 0; ok && i < tiles; ++i, ++j) {
          // K is there, and the weights of the last tile but one have left the columns of its S
          ok = __all_sync(kFull, wait_for(k_full(j), phase(j), fail) && (j < 2 || wait_for(o_done(j), phase(j - 2), fail)));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d = tm + uint32_t(L::S + (j & 1) * TN);
            const uint64_t k0 = smem_desc_sw128(L::K0 + uint32_t(j & 1) * 0x8000u);
            if (few) {
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                  tc_mma_f16(d, k0 + uint64_t(((ks >> 2) * (TN * 128) + (ks & 3) * 32) >> 4),
                             smem_desc_sw128(L::QB) + uint64_t(((part * (D / 64) + (ks >> 2)) * 2048 + (ks & 3) * 32) >> 4),
                             L::idesc(16), uint32_t(part + ks > 0));
            } else {
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                  const uint64_t k = k0 + uint64_t(((ks >> 2) * (TN * 128) + (ks & 3) * 32) >> 4);
                  if (D > 128 && part)
                    tc_mma_f16(d, smem_desc_sw128(L::qlow(ks >> 2)) + uint64_t(((ks & 3) * 32) >> 4), k, L::idesc(TN), 1u);
                  else
                    tc_mma_f16_ts(d, tm + uint32_t((part ? L::QL : L::Q) + 8 * ks), k, L::idesc(TN), uint32_t(part + ks > 0));
                }
            }
            mma_commit(s_full(j));
          }
          __syncwarp();
        }
      } else {
        for (int i = 0; ok && i < tiles; ++i, ++j) {
          ok = __all_sync(kFull, wait_for(v_full(j), phase(j), fail) && wait_for(p_full(j), phase(j), fail));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t p = tm + uint32_t(L::S + (j & 1) * TN);
            const uint64_t v0 = smem_desc_mn128(L::VT, TN * 128);  // 16 tokens per step of 2 KB
            if (few) {  // for d = 64 the product's rows past 64 are not read
              const uint64_t pt = smem_desc_sw128(L::PT + uint32_t(j & 1) * 4096);
#pragma unroll
              for (int ks = 0; ks < TN / 16; ++ks)
                tc_mma_f16(tm + uint32_t(L::O), v0 + uint64_t(ks * 128), pt + uint64_t(((ks >> 2) * 2048 + (ks & 3) * 32) >> 4),
                           L::idesc(16) | (1u << 15), uint32_t(i > 0 || ks > 0));
            } else {
#pragma unroll
              for (int ks = 0; ks < TN / 16; ++ks)
                tc_mma_f16_ts(tm + uint32_t(L::O), p + uint32_t(ks < TN / 32 ? 8 * ks : TN / 4 + 8 * ks), v0 + uint64_t(ks * 128),
                              L::idesc(D) | (1u << 16), uint32_t(i > 0 || ks > 0));
            }
            mma_commit(o_done(j));
          }
          __syncwarp();
        }
      }
    }
    // products still in flight end before the tensor memory is given up
    uint64_t* drain = &bars[o_side ? 16 : 11];
    if (elect_one()) {
      mbar_init(drain, 1);
      fence_mbarrier_init();
      mma_commit(drain);
    }
    __syncwarp();
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

template <int D> cudaError_t launch_tc(const SharedArgs& a, cudaStream_t stream) {
  auto k = shared_tc_kernel<D>;
  static std::atomic<uint64_t> done;
  const cudaError_t e = allow_kernel(k, int(Tc<D>::kTotal), &done);
  if (e != cudaSuccess) return e;
  SharedMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  const int64_t tokens[2] = {a.prefix, a.batch * a.cap};
  for (int p = 0; p < 2; ++p) {
    if (tokens[p] == 0) continue;
    if (D * a.k_bits / 8 % 16 == 0 &&
        !head_rows_tensor_map(&maps.k[p], a.k_codes[p], tokens[p], a.hkv, D * a.k_bits / 8, Tc<D>::PR))
      return cudaErrorNotSupported;
    if (D * a.v_bits / 8 % 16 == 0 &&
        !head_rows_tensor_map(&maps.v[p], a.v_codes[p], tokens[p], a.hkv, D * a.v_bits / 8, Tc<D>::PR))
      return cudaErrorNotSupported;
  }
  return launch_pdl(k, dim3(unsigned(a.grid)), dim3(kThreads), Tc<D>::kTotal, stream, a, maps);
}

}  // namespace

cudaError_t launch_shared_tc(const SharedArgs& a, cudaStream_t stream) {
  int dev = 0, reserved = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e != cudaSuccess) return e;
  if (uint32_t(reserved) != Tc<128>::kBase) return cudaErrorNotSupported;
  if (a.d == 64) return launch_tc<64>(a, stream);
  return a.d == 128 ? launch_tc<128>(a, stream) : launch_tc<256>(a, stream);
}

}  // namespace rrq
