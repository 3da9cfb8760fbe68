// What the softmax cross entropy's files share.
#pragma once
#include "tile.h"
#include "training.h"

namespace cutbce {

namespace {

__host__ __device__ constexpr inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
template <typename T> __device__ inline T* at(char* base, size_t off) { return (T*)(base + off); }

// c, and the sign that H takes: a scale of 0 (or one too small) makes H 0.
__device__ inline float base2(float scale) {
  const float c = fabsf(scale) * kLog2e;
  return c > 0.f ? c : 1.f;
}

// Units of work of the sweep over the vocabulary: tiles of sweep_rows(D) rows x shares of its stages of kSweepStage items. The
// resident workgroups (one a CU, two of narrow rows) take units in turn, kSweepUnits at most: of the numbers of shares
// that make one unit each, two, ... the first is taken that leaves at most 4% of them idle in the last turn, or the best.
constexpr int kSweepStage = 64, kSweepUnits = 1024;
__host__ __device__ constexpr inline int sweep_rows(int D) { return D <= 128 ? 256 : 128; }
__host__ __device__ constexpr inline int sweep_grid(int D) { return D <= 64 ? 512 : 256; }
__host__ __device__ inline int sweep_shares(int64_t tiles, int64_t stages, int grid) {
  const int64_t most = stages / 4 < 1 ? 1 : stages / 4;
  int64_t best = 1;
  float good = 0.f;
  for (int units = grid; units <= kSweepUnits; units += grid) {
    int64_t s = tiles ? units / tiles : 1;
    s = s < 1 ? 1 : (s > most ? most : s);
    const float e = (float)(tiles * s) / (float)(grid * cdiv(tiles * s, grid));
    if (e > good) good = e, best = s;
    if (e >= 0.96f) break;
  }
  return (int)best;
}

}  // namespace

}  // namespace cutbce
