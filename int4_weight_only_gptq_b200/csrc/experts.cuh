// The rows of a mixture-of-experts product as its kernels see them: sorted by
// expert, expert e's rows being offsets[e] .. offsets[e + 1] - 1, with the
// offsets known on the device only.  Each CTA turns them into token tiles of
// its own kernel's size in shared memory.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace gptq {

// One token tile: `rows` rows of expert `e` from row `row0` on, multiplied
// with an MMA width of `n` >= rows.
struct ExpertTile {
  int e, row0, rows, n;
};

// Per expert its first row, its rows and its first token tile (tiles of all
// experts numbered one after another; tile[E] is their number).  An expert's
// rows are spread evenly over its tiles: with a fixed weight tile to
// dequantise per token tile, two half-full tiles cost less than a full one
// and a nearly empty one.  STEP: the MMA width comes in multiples of it;
// MAX_N: the largest width.
template <int MAX_N, int STEP>
struct ExpertTable {
  int* row;   // [E]
  int* rows;  // [E]
  int* tile;  // [E + 1]
  int E;

  static constexpr int bytes(int E) { return 4 * (3 * E + 1); }

  __device__ void place(void* smem, int experts) {
    E = experts;
    row = static_cast<int*>(smem);
    rows = row + E;
    tile = rows + E;
  }

  __device__ static int width(int rows) {
    const int tiles = (rows + MAX_N - 1) / MAX_N;
    const int even = (rows + tiles - 1) / tiles;
    return (even + STEP - 1) / STEP * STEP;
  }

  // Called by every thread of the CTA (`threads` of them).  Offsets outside
  // 0 .. R or not ascending are clamped, so that no row outside the tensors
  // is touched, and reported; the work stays that of R rows.
  __device__ void build(const int32_t* offsets, int R, int threads, int* err) {
    for (int e = threadIdx.x; e < E; e += threads) {
      const int a = offsets[e], b = offsets[e + 1];
      const int lo = min(max(a, 0), R), hi = min(max(b, lo), R);
      if (a != lo || b != hi) atomicCAS(err, 0, kDeviceErrIndex);
      const int c = hi - lo;
      row[e] = lo;
      rows[e] = c;
      const int w = c > 0 ? width(c) : 1;
      tile[e] = (c + w - 1) / w;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      int before = 0;
      for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + (int)threadIdx.x;
        const int c = e < E ? tile[e] : 0;
        int s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, s, o);
          if ((int)threadIdx.x >= o) s += v;
        }
        if (e < E) tile[e] = before + s - c;
        before += __shfl_sync(0xffffffffu, s, 31);
      }
      // (offsets that overlap give more tiles than R rows can have)
      if (threadIdx.x == 0) tile[E] = min(before, min(R, E + R / MAX_N));
    }
    __syncthreads();
  }

  __device__ int tiles() const { return tile[E]; }

  // Token tile t (0 <= t < tiles()).
  __device__ ExpertTile find(int t) const {
    int lo = 0, hi = E;  // tile[lo] <= t < tile[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int w = width(rows[lo]), at = (t - tile[lo]) * w, r = min(w, rows[lo] - at);
    return ExpertTile{lo, row[lo] + at, r, (r + STEP - 1) / STEP * STEP};
  }
};

}  // namespace gptq
