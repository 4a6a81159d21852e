// Rows of a serving batch that name the same state of a pool (gfx950).
#pragma once
#include "common.hpp"

namespace ttt {

// The first position >= from of `slot` in slots[0, rows), or rows: blocks of 512 that do not hold it are passed over at
// two loads a lane (4096 rows of 32 heads: 3.76 ms; all of them by 64 slots a time 6.17), the rest goes by 64.
__device__ __forceinline__ int next_row(const int32_t* slots, int rows, int from, int slot) {
  const int lane = threadIdx.x & 63;
  int at = from;
  for (; at + 512 <= rows; at += 512) {
    int4 s[2];
    bool in = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) __builtin_memcpy(&s[i], slots + at + i * 256 + lane * 4, 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) in |= s[i].x == slot | s[i].y == slot | s[i].z == slot | s[i].w == slot;
    if (__ballot(in)) break;
  }
  for (; at < rows; at += 64) {
    const unsigned long long hit = __ballot(at + lane < rows && slots[at + lane < rows ? at + lane : from] == slot);
    if (hit) return at + __builtin_ctzll(hit);
  }
  return rows;
}

}  // namespace ttt
