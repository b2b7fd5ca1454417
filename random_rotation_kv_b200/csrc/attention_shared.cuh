// attention_shared.cuh — device side of the shared-prefix attention's schedule
// (attention_shared.h), and the code reader its kernels share.
#pragma once

#include "attention_shared.h"
#include "rrq_device.cuh"

namespace rrq {

// A run of tiles of one unit inside one range.
struct Segment {
  int part;            // 0: prefix, 1: tail
  int g;               // kv head
  int b;               // sequence (tails), row tile (prefix)
  int nrows;           // query rows
  int tiles;
  int64_t row0;        // first query row of the unit
  int64_t token_base;  // cache row of token 0 of the unit, over hkv
  int64_t t0, t1;      // tokens [t0, t1)
  int64_t state;       // row of SharedArgs::stats / acc that belongs to the unit's row 0
};

__device__ __forceinline__ int shared_ptotal(const SharedArgs& a) { return a.hkv * a.row_tiles * a.ptiles; }

// The last sequence whose tail begins at or before `x`, by tiles (COST false: x tiles of
// one kv head times hkv behind the prefix) or by cost.
template <bool COST> __device__ __forceinline__ int64_t tail_before(const SharedArgs& a, int64_t x) {
  int64_t lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    const int4 e = a.tails[mid];
    const int64_t at = COST ? int64_t(a.hkv) * (int64_t(e.x) * a.tcost + int64_t(e.y) * a.scost) : int64_t(a.hkv) * e.x;
    if (at <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
// Cost before the first tile of the tail of sequence entry `e` at kv head g, and the range a tile of
// that cost belongs to.
__device__ __forceinline__ int64_t tail_cost(const SharedArgs& a, const int4& e, int g) {
  return int64_t(shared_ptotal(a)) * a.pcost + (int64_t(a.hkv) * e.x + int64_t(g) * e.w) * a.tcost +
         (int64_t(a.hkv) * e.y + g) * a.scost;
}
__device__ __forceinline__ int range_of_cost(const SharedArgs& a, int64_t cost) { return int(cost / a.head[1]); }

// The first tile of the line whose cost is at least `cost`.
__device__ __forceinline__ int tile_at_cost(const SharedArgs& a, int64_t cost) {
  const int ptotal = shared_ptotal(a), total = a.head[0];
  const int64_t p = int64_t(ptotal) * a.pcost;
  if (cost <= p) return int((cost + a.pcost - 1) / a.pcost);
  if (total == ptotal) return total;
  const int64_t x = cost - p, b = tail_before<true>(a, x);
  const int4 e = a.tails[b];
  const int64_t y = x - int64_t(a.hkv) * (int64_t(e.x) * a.tcost + int64_t(e.y) * a.scost);
  if (e.w == 0) return total;  // behind the last tile
  const int64_t unit = int64_t(e.w) * a.tcost + a.scost, g = y / unit;
  if (g >= a.hkv) return total;
  const int64_t i = (y - g * unit + a.tcost - 1) / a.tcost;
  const int64_t t = ptotal + int64_t(a.hkv) * e.x + g * e.w + (i < e.w ? i : e.w);
  return int(t < total ? t : total);
}
__device__ __forceinline__ void range_tiles(const SharedArgs& a, int range, int* pos, int* end) {
  *pos = tile_at_cost(a, int64_t(range) * a.head[1]);
  *end = tile_at_cost(a, int64_t(range + 1) * a.head[1]);
}

// Fills the unit's fields of a segment from its kv head and row tile or sequence entry.
__device__ __forceinline__ void prefix_unit(const SharedArgs& a, int g, int rt, Segment* s) {
  s->part = 0;
  s->g = g;
  s->b = rt;
  s->row0 = int64_t(rt) * 128;
  s->nrows = int(a.rows - s->row0 < 128 ? a.rows - s->row0 : 128);
  s->token_base = 0;
}
__device__ __forceinline__ void tail_unit(const SharedArgs& a, int g, int64_t b, Segment* s) {
  s->part = 1;
  s->g = g;
  s->b = int(b);
  s->row0 = b * a.group;
  s->nrows = a.group;
  s->token_base = b * a.cap;
}
// Tokens and state of the segment that starts at tile `at` of a unit of `tiles` tiles and
// `len` tokens, `left` tiles before its range's end; it is the unit's part number `part`.
__device__ __forceinline__ void cut_segment(const SharedArgs& a, int at, int tiles, int64_t len, int left, int part, Segment* s) {
  s->tiles = tiles - at < left ? tiles - at : left;
  s->t0 = int64_t(at) * a.tile;
  const int64_t t1 = s->t0 + int64_t(s->tiles) * a.tile;
  s->t1 = t1 < len ? t1 : len;
  s->state = (int64_t(part + (s->part ? a.parts_p : 0)) * a.hkv + s->g) * a.rows + s->row0;
}

// The segment at position `pos` of the line (pos < end, the range's end).
__device__ __forceinline__ Segment segment_at(const SharedArgs& a, int range, int pos, int end) {
  Segment s;
  const int ptotal = shared_ptotal(a);
  if (pos < ptotal) {
    const int u = pos / a.ptiles;
    prefix_unit(a, u / a.row_tiles, u % a.row_tiles, &s);
    cut_segment(a, pos - u * a.ptiles, a.ptiles, a.prefix, end - pos,
                range - range_of_cost(a, int64_t(u) * a.ptiles * a.pcost), &s);
  } else {
    const int x = pos - ptotal;
    const int64_t b = tail_before<false>(a, x);  // the last entry at or before x is not empty
    const int4 e = a.tails[b];
    const int in = x - a.hkv * e.x, g = in / e.w;
    tail_unit(a, g, b, &s);
    cut_segment(a, in - g * e.w, e.w, e.z, end - pos, range - range_of_cost(a, tail_cost(a, e, g)), &s);
  }
  return s;
}

// The b-bit codes of 8 coordinates (b bytes at `p`) as one 4-bit code per nibble.
__device__ __forceinline__ uint32_t octet_nibbles(uint32_t w, int bits) {
  if (bits == 4) return w;
  if (bits == 3) {
    w = (w & 0xfffu) | ((w & 0xfff000u) << 4);
    w = (w & 0x003f003fu) | ((w & 0x0fc00fc0u) << 2);
    return (w & 0x07070707u) | ((w & 0x38383838u) << 1);
  }
  if (bits == 2) {
    w = (w & 0xffu) | ((w & 0xff00u) << 8);
    w = (w & 0x000f000fu) | ((w & 0x00f000f0u) << 4);
    return (w & 0x03030303u) | ((w & 0x0c0c0c0cu) << 2);
  }
  w = (w & 0x0fu) | ((w & 0xf0u) << 12);
  w = (w & 0x00030003u) | ((w & 0x000c000cu) << 6);
  return (w & 0x01010101u) | ((w & 0x02020202u) << 3);
}

}  // namespace rrq
