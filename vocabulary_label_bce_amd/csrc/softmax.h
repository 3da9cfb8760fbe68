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
__host__ __device__ constexpr inline int sweep_stages(int64_t V) { return (int)(((uint32_t)V + kSweepStage - 1) / kSweepStage); }
__host__ __device__ constexpr inline int sweep_rows(int D) { return D <= 128 ? 256 : 128; }
__host__ __device__ constexpr inline int sweep_grid(int D) { return D <= 64 ? 512 : 256; }
__host__ __device__ inline int sweep_shares(int tiles, int stages, int grid) {  // (32 bits: these are quotients)
  const int most = stages / 4 < 1 ? 1 : stages / 4;
  int best = 1;
  float good = 0.f;
  for (int units = grid; units <= kSweepUnits; units += grid) {
    int s = tiles ? units / tiles : 1;
    s = s < 1 ? 1 : (s > most ? most : s);
    const float e = (float)(tiles * s) / (float)(grid * ((tiles * s + grid - 1) / grid));
    if (e > good) good = e, best = s;
    if (e >= 0.96f) break;
  }
  return best;
}
// Steps first .. first + count - 1 of `steps` are share `share` of `shares`: the first steps % shares have one more.
struct Share {
  int first, count;
};
__device__ inline Share share_at(int steps, int shares, int share) {
  const int each = steps / shares, more = steps - each * shares;
  return {share * each + (share < more ? share : more), each + (share < more ? 1 : 0)};
}

// Joining a row's shares, (reference, sum of exponentials): the largest reference of a share in which something counts
// (one in which nothing does has the sum 0, whatever its reference), a share's factor, and what is kept of a row.
__device__ inline float top_of(float m, float2 share) { return share.y == 0.f ? m : fmaxf(m, share.x); }
__device__ inline float share_of(float2 share, float m) { return share.y == 0.f ? 0.f : exp2_of(share.x - m); }
__device__ inline void finish_row(const Ce& c, int i, int64_t r, float z, float m, float others, float* row_loss,
                                  float* each) {
  const float mine = exp2_of(z - m), sum = others + mine;
  const float l = mine == 1.f ? log1pf(others) : (m - z) * kLn2 + logf(sum);
  const float coef = at<float>(c.saved, c.at.coef)[i];
  at<float>(c.saved, c.at.shift)[i] = m + log2f(sum) - log2f(coef);
  at<float>(c.saved, c.at.own)[i] = -coef * (others / sum);
  each[i] = l;
  if (row_loss) row_loss[r] = l;
}

}  // namespace

}  // namespace cutbce
