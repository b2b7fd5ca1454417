// attention_shared.cu — one decode step of attention for a batch of sequences over a
// shared quantised prefix and a private quantised tail each.
//
// With g the kv head of query head h, over the prefix and then the sequence's tail:
//     out = Σ_t p_t·v̂_t,   p = softmax(scale·⟨q, k̂_t⟩),   k̂ = Πᵀ(ν/√d·c[code]),
// and Πᵀ = D·H/√d, so with q' = scale·log2 e/d · H·D·q the base-2 score is
// x_t = ν_t·⟨q', c[code_t]⟩, the values are summed in their rotated domain and
// rotated back once per row: out = D·H·(Σ 2^{x_t − m}·ν_t·c[code_t]) / (d·Σ 2^{x_t − m}).
//
// Three launches: the queries are rotated (and the tails' tiles counted), every CTA walks
// its range of the line of tiles (attention_shared.h) and leaves a partial state
// (m, Σ 2^{x − m}, Σ 2^{x − m}·ν·c) per unit, and one warp per query row merges its parts
// and rotates back.  No CTA waits for another, and nothing depends on the order in which
// they run.
#include <cmath>

#include "attention_shared.cuh"

namespace rrq {
namespace {

constexpr int kTcMaxD = 256;  // head sizes of the tensor-core kernel
constexpr int kMinTiles = 2;  // tiles per range at least: a state costs about as much as a tile

// Walsh–Hadamard transform over a warp's row: coordinate 32·i + lane in v[i].
template <int N> __device__ __forceinline__ void fwht_row(float (&v)[N], int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float o = __shfl_xor_sync(kFull, v[i], m);
      v[i] = lane & m ? o - v[i] : v[i] + o;
    }
#pragma unroll
  for (int m = 1; m < N; m <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & m)) {
        const float x = v[i], y = v[i | m];
        v[i] = x + y;
        v[i | m] = x - y;
      }
}

// ---- the line of tiles, by one block of 256 threads.  A unit's parts are the ranges that
// its tiles' costs fall into; part in range r of the U-th non-empty unit is segment U + r,
// as each range before r adds at most one segment to those of the units before.  All costs
// are below 2^30.
__device__ __forceinline__ void put_segment(const SharedArgs& a, int index, const SharedSegment& s) {
  a.segs[2 * index] = make_int4(s.token, s.tokens, s.tiles, s.g);
  a.segs[2 * index + 1] = make_int4(s.row0, s.nrows, s.state, s.flags);
}
// Tiles [at, end) of a unit of `tokens` tokens (its token 0 in s.token) as part `part`.
__device__ __forceinline__ void put_part(const SharedArgs& a, int index, SharedSegment s, int at, int end, int tokens, int part,
                                         bool last) {
  s.token += at * a.tile;
  s.tokens = (end * a.tile < tokens ? end * a.tile : tokens) - at * a.tile;
  s.tiles = end - at;
  s.state = part * a.hkv + s.g;
  s.flags |= last ? 2 : 0;
  put_segment(a, index, s);
}

__device__ void lay_out(const SharedArgs& a) {
  __shared__ int2 s_sum[8];
  __shared__ int4 s_tail[256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int r = tid; r < a.grid; r += 256) a.begin[r] = -1;  // the barrier below comes before the others' entries
  // tokens and tiles of a sequence's tail
  auto length = [&](int64_t b) {
    if (b >= a.batch || a.lens == nullptr) return 0;
    const int n = a.lens[b];
    return n < 0 ? 0 : n > a.cap ? int(a.cap) : n;
  };
  // all tails' tiles and how many are not empty
  int tiles = 0, filled = 0;
  for (int64_t b = tid; b < a.batch; b += 256) {
    const int n = (length(b) + a.tile - 1) / a.tile;
    tiles += n;
    filled += n > 0;
  }
  tiles = __reduce_add_sync(kFull, tiles);
  filled = __reduce_add_sync(kFull, filled);
  if (lane == 0) s_sum[warp] = make_int2(tiles, filled);
  __syncthreads();
  tiles = filled = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) tiles += s_sum[w].x, filled += s_sum[w].y;
  const int pcost = a.units_p * a.ptiles * a.pcost;
  const int cost = pcost + a.hkv * (tiles * a.tcost + filled * a.scost);
  const int even = (cost + a.grid - 1) / a.grid;
  const int per = even < a.min_cost ? a.min_cost : even;
  const int units = a.units_p + a.hkv * filled;
  // the prefix, a thread per range: its tiles of one prefix unit after the other
  const int ptotal = a.units_p * a.ptiles;
  for (int r = tid; r < a.grid && ptotal > 0; r += 256) {
    int pos = (r * per + a.pcost - 1) / a.pcost, end = ((r + 1) * per + a.pcost - 1) / a.pcost;
    if (end > ptotal) end = ptotal;
    const bool more = units > a.units_p && pcost / per == r;  // the first tail begins in this range
    if (pos < end) a.begin[r] = pos / a.ptiles + r;
    while (pos < end) {
      const int u = pos / a.ptiles, at = pos - u * a.ptiles;
      const int to = end - u * a.ptiles < a.ptiles ? end - u * a.ptiles : a.ptiles;
      SharedSegment s = {};
      s.g = u / a.row_tiles;
      s.row0 = (u - s.g * a.row_tiles) * 128;
      s.nrows = int(a.rows - s.row0 < 128 ? a.rows - s.row0 : 128);
      const int r0 = u * a.ptiles * a.pcost / per;
      pos += to - at;
      put_part(a, u + r, s, at, to, int(a.prefix), r - r0, pos == end && !more);
      if (to == a.ptiles) a.counts[u] = r - r0 + 1;
    }
  }
  // the tails, a thread per sequence and kv head
  int before = 0, some_before = 0;
  for (int64_t b0 = 0; b0 < a.batch && a.cap > 0; b0 += 256) {
    const int64_t b = b0 + tid;
    const int len = length(b), mine = (len + a.tile - 1) / a.tile;
    int sum = mine, some = mine > 0;  // inclusive prefixes: of the warp, then of the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, sum, o), y = __shfl_up_sync(kFull, some, o);
      if (lane >= o) sum += x, some += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = make_int2(sum, some);
    __syncthreads();
    int all = 0, all_some = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const int2 x = s_sum[w];
      if (w < warp) sum += x.x, some += x.y;
      all += x.x;
      all_some += x.y;
    }
    s_tail[tid] = make_int4(before + sum - mine, some_before + some - (mine > 0), len, mine);
    before += all;
    some_before += all_some;
    __syncthreads();
    const int here = int(a.batch - b0 < 256 ? a.batch - b0 : 256) * a.hkv;
    for (int k = tid; k < here; k += 256) {
      const int bb = k / a.hkv, g = k - bb * a.hkv;
      const int4 t = s_tail[bb];  // tiles and non-empty tails before it, tokens, tiles
      int* count = a.counts + a.units_p + b0 * a.hkv + k;
      if (t.w == 0) {
        *count = 0;
        continue;
      }
      SharedSegment s = {};
      s.token = int((b0 + bb) * a.cap);
      s.g = g;
      s.row0 = int((b0 + bb) * a.group);
      s.nrows = a.group;
      s.flags = 1;
      const int unit = a.units_p + a.hkv * t.y + g;
      const int from = pcost + (a.hkv * t.x + g * t.w) * a.tcost + (a.hkv * t.y + g) * a.scost;
      const int r0 = from / per, r1 = (from + (t.w - 1) * a.tcost) / per;
      const int rn = unit + 1 < units ? (from + t.w * a.tcost + a.scost) / per : -1;  // the next unit's first range
      int done = 0;
      for (int r = r0; r <= r1; ++r) {
        const int end = r == r1 ? t.w : ((r + 1) * per - from + a.tcost - 1) / a.tcost;
        put_part(a, unit + r, s, done, end, t.z, a.parts_p + r - r0, r < r1 || rn != r);
        if (r > r0 || unit == 0) a.begin[r] = unit + r;
        done = end;
      }
      // a range that begins with this unit or with the next one
      if (unit == a.units_p && unit > 0 && (pcost - a.pcost) / per < r0) a.begin[r0] = unit + r0;
      if (rn > r1) a.begin[rn] = unit + 1 + rn;
      *count = r1 - r0 + 1;
    }
    __syncthreads();
  }
}

// ---- queries rotated, one warp per row; one block more lays out the line of tiles
template <int D>
__global__ void __launch_bounds__(256) shared_prepare_kernel(const SharedArgs a) {
  constexpr int N = D / 32;
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0) {
    lay_out(a);
    return;
  }
  const int64_t row = int64_t(blockIdx.x - 1) * 8 + warp;  // b·hq + h
  if (row >= a.batch * a.hq) return;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t at = row * D + 32 * i + lane;
    const float x = a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at])
                           : __half2float(static_cast<const __half*>(a.q)[at]);
    v[i] = sign_bit(a.k_seed, 32 * i + lane) ? -x : x;
  }
  fwht_row(v, lane);
  const int64_t b = row / a.hq;
  const int h = int(row % a.hq), g = h / a.group;
  const int64_t to = int64_t(g) * a.rows + b * a.group + h % a.group;
  if constexpr (D > kTcMaxD) {
#pragma unroll
    for (int i = 0; i < N; ++i) a.qrot[to * D + 32 * i + lane] = v[i] * a.kscale;
  } else {
    // fp16, the row's largest magnitude brought into [2^14, 2^15)
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] *= a.kscale;
      big = fmaxf(big, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
    int e = int(__float_as_uint(big) >> 23) - 127;
    if (e < -100) e = -100;
    const float f = __uint_as_float(uint32_t(127 + 14 - e) << 23);
    if (lane == 0) a.qexp[to] = __uint_as_float(uint32_t(127 + e - 14) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = v[i] * f;
      const __half hi = __float2half_rn(x);
      a.qh[to * D + 32 * i + lane] = hi;
      a.ql[to * D + 32 * i + lane] = __float2half_rn(x - __half2float(hi));
    }
  }
}

// ---- partial states: 8 query rows at a time, one warp each, 32 tokens per step
template <int D>
__global__ void __launch_bounds__(256) shared_partial_kernel(const SharedArgs a) {
  constexpr int N = D / 32, P = D + 1;
  extern __shared__ float sm[];
  float* s_kv = sm;             // [32][P] values of 32 tokens
  float* s_q = sm + 32 * P;     // [8][D]
  float* s_lev = s_q + 8 * D;   // [2][16]
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 16) s_lev[tid] = a.k_levels[tid];
  else if (tid < 32) s_lev[tid] = a.v_levels[tid - 16];
  const int range = blockIdx.x;
  for (int i = a.begin[range]; i >= 0;) {
    const SharedSegment s = shared_segment(a, i);
    i = s.flags & 2 ? -1 : i + 1;
    const int kv = s.flags & 1;
    const int64_t state = int64_t(s.state) * a.rows + s.row0;
    // 32 tokens' values (codes' levels, unscaled) into s_kv; tokens past the end repeat the last
    auto load = [&](const uint8_t* codes, int bits, const float* lev, int64_t t) {
      for (int i = tid; i < 32 * (D / 8); i += 256) {
        const int tok = i / (D / 8), o = i % (D / 8);
        const int64_t tt = t + tok < s.tokens ? t + tok : s.tokens - 1;
        const uint8_t* p = codes + ((s.token + tt) * a.hkv + s.g) * (D * bits / 8) + o * bits;
        uint32_t w = 0;
        for (int k = 0; k < bits; ++k) w |= uint32_t(p[k]) << (8 * k);
        w = octet_nibbles(w, bits);
        for (int j = 0; j < 8; ++j) s_kv[tok * P + 8 * o + j] = lev[(w >> (4 * j)) & 15u];
      }
    };
    for (int r0 = 0; r0 < s.nrows; r0 += 8) {
      const int r = r0 + warp;
      const bool live = r < s.nrows;
      const float* q = a.qrot + (int64_t(s.g) * a.rows + s.row0 + (live ? r : 0)) * D;
      for (int i = lane; i < D; i += 32) s_q[warp * D + i] = q[i];
      float m = -INFINITY, l = 0.f, acc[N];
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
      for (int64_t t = 0; t < s.tokens; t += 32) {
        __syncthreads();
        load(a.k_codes[kv], a.k_bits, s_lev, t);
        __syncthreads();
        const bool valid = t + lane < s.tokens;
        const int64_t row = (s.token + (valid ? t + lane : s.tokens - 1)) * a.hkv + s.g;
        float x = 0.f;
        for (int i = 0; i < D; ++i) x = fmaf(s_q[warp * D + i], s_kv[lane * P + i], x);
        x = valid ? x * a.k_norms[kv][row] : -INFINITY;
        const float nu = a.v_norms[kv][row];
        float mx = x;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        const float mn = fmaxf(m, mx), f = exp2f(m - mn);
        const float p = valid ? exp2f(x - mn) : 0.f;
        m = mn;
        l = l * f + p;
        for (int i = 0; i < N; ++i) acc[i] *= f;
        const float w = valid ? p * nu : 0.f;
        __syncthreads();
        load(a.v_codes[kv], a.v_bits, s_lev + 16, t);
        __syncthreads();
        for (int k = 0; k < 32; ++k) {
          const float wk = __shfl_sync(kFull, w, k);
          for (int i = 0; i < N; ++i) acc[i] = fmaf(wk, s_kv[k * P + 32 * i + lane], acc[i]);
        }
      }
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
      if (live) {
        if (lane == 0) a.stats[state + r] = make_float2(m, l);
        for (int i = 0; i < N; ++i) a.acc[(state + r) * D + 32 * i + lane] = acc[i];
      }
      __syncthreads();
    }
  }
}

// ---- W warps per query row: its parts merged, rotated back, rounded to the output type.  Each
// warp takes every W-th part; with W = 8 (calls of few rows, where latency counts) the
// warps' sums meet in shared memory.
template <int D, int W>
__global__ void __launch_bounds__(256) shared_merge_kernel(const SharedArgs a) {
  constexpr int N = D / 32;
  __shared__ float s_sum[W > 1 ? W : 1][W > 1 ? D : 1], s_l[8];
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = W > 1 ? warp : 0;
  const int64_t row = W > 1 ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + warp;  // b·hq + h
  if (row >= a.batch * a.hq) return;
  const int64_t b = row / a.hq;
  const int h = int(row - b * a.hq), g = h / a.group;
  const int64_t r = b * a.group + h % a.group;
  // parts of the prefix, of the tail
  const int np = a.units_p > 0 ? a.counts[g * a.row_tiles + int(r / 128)] : 0;
  const int nt = a.cap > 0 ? a.counts[a.units_p + b * a.hkv + g] : 0;
  auto state = [&](int i) {
    const int p = i < np ? i : a.parts_p + (i - np);
    return (int64_t(p) * a.hkv + g) * a.rows + r;
  };
  const int n = np + nt;
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, a.stats[state(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  // lane i takes part mine + W·i; the parts' sums come in batches of independent loads
  constexpr int kBatch = W > 1 ? 4 : N <= 4 ? 8 : 4;
  float v[N], l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int i0 = mine; i0 < n; i0 += 32 * W) {
    float f = 0.f;
    int64_t st = state(i0);
    const int i = i0 + lane * W;
    if (i < n) {
      st = state(i);
      const float2 ml = a.stats[st];
      f = exp2f(ml.x - m);
      l = fmaf(ml.y, f, l);
    }
    const int left = (n - i0 + W - 1) / W, here = left < 32 ? left : 32;
    for (int k0 = 0; k0 < here; k0 += kBatch) {
      float x[kBatch][N], fk[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int from = k0 + k < here ? k0 + k : 0;
        const int64_t at = __shfl_sync(kFull, st, from) * D + lane;
        fk[k] = __shfl_sync(kFull, f, from);
        if (k0 + k >= here) fk[k] = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) x[k][e] = k0 + k < here ? a.acc[at + 32 * e] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = fmaf(x[k][e], fk[k], v[e]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < N; ++e) s_sum[warp][32 * e + lane] = v[e];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (warp != 0) return;
    l = s_l[0];
#pragma unroll
    for (int w = 1; w < W; ++w) l += s_l[w];
#pragma unroll
    for (int e = 0; e < N; ++e) {
#pragma unroll
      for (int w = 1; w < W; ++w) v[e] += s_sum[w][32 * e + lane];
    }
  }
  fwht_row(v, lane);
  const float inv = n > 0 ? 1.f / l / (float(D) * a.v_alpha) : 0.f;  // l itself may be near fp32's end
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = 32 * k + lane;
    const float y = n > 0 ? (sign_bit(a.v_seed, c) ? -v[k] : v[k]) * inv : 0.f;
    if (a.bf16) static_cast<__nv_bfloat16*>(a.out)[row * D + c] = __float2bfloat16_rn(y);
    else static_cast<__half*>(a.out)[row * D + c] = __float2half_rn(y);
  }
}

int sm_count() {
  int dev = 0, sms = kSms;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms < 1 ? 1 : sms;
}

template <int D> cudaError_t launch_d(const SharedArgs& a, cudaStream_t stream) {
  const int64_t rows = a.batch * a.hq;
  const dim3 blocks(unsigned((rows + 7) / 8));
  cudaError_t e = launch_pdl(shared_prepare_kernel<D>, dim3(blocks.x + 1), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  if constexpr (D > kTcMaxD) {
    constexpr size_t smem = (32 * (D + 1) + 8 * D + 32) * 4;
    e = cudaFuncSetAttribute(shared_partial_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(shared_partial_kernel<D>, dim3(unsigned(a.grid)), dim3(256), smem, stream, a);
  } else {
    e = launch_shared_tc(a, stream);
  }
  if (e != cudaSuccess) return e;
  // Eight warps per row while that leaves at most six blocks per SM.  Whole calls with eight warps
  // against one: d = 128 at 512 rows 27.9 us against 29.9, 768 rows 32.7 against 33.8, 1024 rows
  // 37.6 against 36.6, 4096 rows 87.1 against 77.2; d = 64 and 256 at 512 rows 21.5 against 22.8 and 29.2
  // against 32.0, at 1152 rows 27.1 against 26.6 and 41.0 against 39.8.
  if (rows <= int64_t(a.grid) * 6) return launch_pdl(shared_merge_kernel<D, 8>, dim3(unsigned(rows)), dim3(256), 0, stream, a);
  return launch_pdl(shared_merge_kernel<D, 1>, blocks, dim3(256), 0, stream, a);
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

bool attention_shared_plan(SharedArgs* a) {
  a->group = a->hq / a->hkv;
  if (a->group > 128) return false;
  a->tile = a->d <= 128 ? 128 : 64;
  const int64_t most = int64_t(1) << 30;  // tiles of all units, in cost
  // a cache's tokens, rounded up to a tile, are counted in 32 bits
  const int64_t tokens = 2 * most - 128;
  if (a->prefix >= tokens || (a->batch > 0 && a->cap >= tokens / a->batch)) return false;
  if (a->prefix / 64 >= most || a->cap / 64 >= most || a->batch >= most / a->hq) return false;
  a->rows = a->batch * a->group;
  a->row_tiles = int((a->rows + 127) / 128);
  const int64_t pt = (a->prefix + a->tile - 1) / a->tile, tt = (a->cap + a->tile - 1) / a->tile;
  const int64_t punits = int64_t(a->hkv) * a->row_tiles, tunits = int64_t(a->hkv) * a->batch;
  if (tunits == 0) return true;  // no sequence: nothing runs
  if (pt > most / punits || tt > most / tunits || (punits * pt + tunits * (tt + 1)) >= most / 10) return false;
  a->ptiles = int(pt);
  a->units_p = pt > 0 ? int(punits) : 0;
  a->grid = sm_count();
  // costs, measured: a tile against up to 16 rows 1.7 us, against more 2.5 us, a tail's start
  // and end 2 us
  a->pcost = a->d <= 128 && a->rows <= 16 ? 7 : 10;
  a->tcost = a->d <= 128 && a->group <= 16 ? 7 : 10;
  a->scost = 8;
  a->min_cost = kMinTiles * 10;
  int64_t per = (punits * pt * a->pcost + a->grid - 1) / a->grid;  // a range is never shorter
  if (per < a->min_cost) per = a->min_cost;
  auto parts = [&](int64_t tiles, int cost) {
    const int64_t p = tiles > 0 ? (tiles - 1) * cost / per + 2 : 0;
    const int64_t most = tiles < a->grid ? tiles : a->grid;  // at least a tile each, one per range
    return int(p < most ? p : most);
  };
  a->parts_p = parts(pt, a->pcost);
  a->parts_t = parts(tt, a->tcost);
  return true;
}

void attention_shared_levels(SharedArgs* a, bool default_k, bool default_v) {
  // by bits: the factor of least mean square error over N(0,1) coordinates, from a search
  // over all fp32 values in [1, 2): relative error 1e-10, 1e-7, 7e-6, 3.8e-5 (2e-4 unscaled)
  static const float kBest[5] = {1.f, 0x1.1dc17p+0f, 0x1.fb2502p+0f, 0x1.24fd4ap+0f, 0x1.429a86p+0f};
  auto alpha = [](const float* lev, int bits, bool dflt) {
    float big = 0.f;
    for (int k = 0; k < 1 << bits; ++k) big = std::fmax(big, std::fabs(lev[k]));
    int e = 0;
    std::frexp(big, &e);  // big in [2^(e − 1), 2^e)
    return dflt ? kBest[bits] : std::ldexp(1.f, e < -99 ? 100 : 1 - e);
  };
  a->k_alpha = a->v_alpha = 1.f;
  if (a->d > kTcMaxD) return;
  a->k_alpha = alpha(a->k_levels, a->k_bits, default_k);
  a->v_alpha = alpha(a->v_levels, a->v_bits, default_v);
  a->kscale /= a->k_alpha;
}

size_t attention_shared_layout(SharedArgs* a, void* base) {
  const size_t rows = size_t(a->rows) * size_t(a->hkv), parts = size_t(a->parts_p) + size_t(a->parts_t);
  const size_t units = size_t(a->units_p) + (a->cap > 0 ? size_t(a->batch) * a->hkv : 0);
  const size_t begin = pad256(size_t(a->grid) * 4), counts = pad256(units * 4), segs = pad256((units + a->grid) * 32);
  const size_t head = begin + counts + segs;
  const size_t q = pad256(rows * a->d * 4), qe = pad256(rows * 4), st = pad256(parts * rows * 8);
  uint8_t* p = static_cast<uint8_t*>(base);
  if (p != nullptr) {
    a->begin = reinterpret_cast<int*>(p);
    a->counts = reinterpret_cast<int*>(p + begin);
    a->segs = reinterpret_cast<int4*>(p + begin + counts);
    a->qrot = reinterpret_cast<float*>(p + head);
    a->qh = reinterpret_cast<__half*>(p + head);
    a->ql = a->qh + rows * a->d;
    a->qexp = reinterpret_cast<float*>(p + head + q);
    a->stats = reinterpret_cast<float2*>(p + head + q + qe);
    a->acc = reinterpret_cast<float*>(p + head + q + qe + st);
  }
  return head + q + qe + st + pad256(parts * rows * a->d * 4);
}

cudaError_t launch_attention_shared(const SharedArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    case 256: return launch_d<256>(a, stream);
    default: return launch_d<512>(a, stream);
  }
}

}  // namespace rrq
