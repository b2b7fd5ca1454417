// attention_shared.cuh — device side of the shared-prefix attention's schedule
// (attention_shared.h), and the code reader its kernels share.
#pragma once

#include "attention_shared.h"
#include "rrq_device.cuh"

namespace rrq {

// A run of tiles of one unit inside one range.
struct SharedSegment {
  int token;   // first token, in rows of its cache over hkv
  int tokens;
  int tiles;
  int g;       // kv head
  int row0;    // first query row of the unit
  int nrows;
  int state;   // part · hkv + g: the unit's row r is row state · rows + row0 + r of stats and acc
  int flags;   // bit 0: a tail (otherwise the prefix), bit 1: the range's last
};
__device__ __forceinline__ SharedSegment shared_segment(const SharedArgs& a, int i) {
  const int4 x = a.segs[2 * i], y = a.segs[2 * i + 1];
  return {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
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
