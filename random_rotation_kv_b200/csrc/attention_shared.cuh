// attention_shared.cuh — device side of the shared-prefix attention's schedule
// (attention_shared.h), and the code reader its kernels share.
#pragma once

#include "attention_shared.h"
#include "rrq_device.cuh"

namespace rrq {

constexpr int kHeadTails = 16;  // first index of the tails' tile sums in SharedArgs::head

__device__ __forceinline__ int shared_tail_len(const SharedArgs& a, int64_t b) {
  const int64_t n = a.lens ? a.lens[b] : 0;
  return int(n < 0 ? 0 : n > a.cap ? a.cap : n);
}

// Cost of the line's first `tile` tiles, the range that tile `tile` belongs to, and a
// range's tiles [*pos, *end): those whose cost begins in it.
__device__ __forceinline__ int64_t shared_cost(const SharedArgs& a, int tile) {
  const int ptotal = a.hkv * a.row_tiles * a.ptiles;
  return tile <= ptotal ? int64_t(tile) * a.pcost : int64_t(ptotal) * a.pcost + int64_t(tile - ptotal) * a.tcost;
}
__device__ __forceinline__ int range_of(const SharedArgs& a, int tile) {
  return int(shared_cost(a, tile) / a.head[1]);
}
__device__ __forceinline__ void range_tiles(const SharedArgs& a, int range, int* pos, int* end) {
  const int total = a.head[0], ptotal = a.hkv * a.row_tiles * a.ptiles;
  auto tile_at = [&](int64_t cost) {
    const int64_t p = int64_t(ptotal) * a.pcost;
    const int64_t t = cost <= p ? (cost + a.pcost - 1) / a.pcost : ptotal + (cost - p + a.tcost - 1) / a.tcost;
    return int(t < total ? t : total);
  };
  *pos = tile_at(int64_t(range) * a.head[1]);
  *end = tile_at(int64_t(range + 1) * a.head[1]);
}

// A run of tiles of one unit inside one range.
struct Segment {
  int part;            // 0: prefix, 1: tail
  int g;               // kv head
  int64_t b;           // sequence (tails)
  int64_t row0;        // first query row of the unit
  int nrows;
  int64_t token_base;  // cache row of token 0 of the unit, over hkv
  int64_t t0, t1;      // tokens [t0, t1)
  int tiles;
  int64_t state;       // row of SharedArgs::stats / acc that belongs to the unit's row 0
};

// The segment at position `pos` of the line (pos < end, the range's end).
__device__ __forceinline__ Segment segment_at(const SharedArgs& a, int range, int pos, int end) {
  Segment s;
  const int ptotal = a.hkv * a.row_tiles * a.ptiles;
  int first, at, unit_tiles;
  int64_t len;
  if (pos < ptotal) {
    const int u = pos / a.ptiles;
    first = u * a.ptiles;
    unit_tiles = a.ptiles;
    s.part = 0;
    s.g = u / a.row_tiles;
    s.b = 0;
    s.row0 = int64_t(u % a.row_tiles) * 128;
    s.nrows = int(a.rows - s.row0 < 128 ? a.rows - s.row0 : 128);
    s.token_base = 0;
    len = a.prefix;
  } else {
    const int* sums = a.head + kHeadTails;
    const int x = pos - ptotal;
    int64_t lo = 0, hi = a.batch;  // the last b with hkv·sums[b] ≤ x: its tail is not empty
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (int64_t(a.hkv) * sums[mid] <= x) lo = mid;
      else hi = mid;
    }
    const int before = sums[lo];
    unit_tiles = sums[lo + 1] - before;
    s.part = 1;
    s.b = lo;
    s.g = (x - a.hkv * before) / unit_tiles;
    first = ptotal + a.hkv * before + s.g * unit_tiles;
    s.row0 = lo * a.group;
    s.nrows = a.group;
    s.token_base = lo * a.cap;
    len = shared_tail_len(a, lo);
  }
  at = pos - first;
  s.tiles = unit_tiles - at < end - pos ? unit_tiles - at : end - pos;
  s.t0 = int64_t(at) * a.tile;
  s.t1 = s.t0 + int64_t(s.tiles) * a.tile < len ? s.t0 + int64_t(s.tiles) * a.tile : len;
  const int p = range - range_of(a, first) + (s.part ? a.parts_p : 0);
  s.state = (int64_t(p) * a.hkv + s.g) * a.rows + s.row0;
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
