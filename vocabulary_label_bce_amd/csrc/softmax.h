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

// Units of work of the sweep over the vocabulary: tiles of sweep_rows(D) rows x shares of its stages of kSweepStage
// items. The resident workgroups (one a CU, two of narrow rows) take units in turn, kSweepUnits at most: of the
// numbers of shares that make one unit each, two, ... the first is taken that leaves at most 4% of them idle in the
// last turn, or the best.
constexpr int kSweepStage = 64, kSweepUnits = 1024;
__host__ __device__ constexpr inline int sweep_stages(int64_t V) {
  return (int)(((uint32_t)V + kSweepStage - 1) / kSweepStage);
}
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

// Joining a row's shares, (reference, sum of exponentials): the largest reference of a share in which something counts,
// a share's factor, and what is kept of a row. A share in which nothing counts has the sum 0 and the reference 0 or
// -inf. Another one has lost its largest exponential, which is 1 but for the reference's rounding: exponents are formed
// by one multiply-add, so that a reference from 2^31 on may be off by 64 and more, and beyond float32 it is infinite.
// Such a share, left out, would leave a loss that looks like one; it makes its row not a number.
__device__ inline bool lost(float2 share) { return share.y == 0.f && share.x != 0.f && share.x != -INFINITY; }
__device__ inline float top_of(float m, float2 share) { return share.y == 0.f ? m : fmaxf(m, share.x); }
__device__ inline float share_of(float2 share, float m) {
  return lost(share) ? NAN : share.y == 0.f ? 0.f : exp2_of(share.x - m);
}
// Probabilities are exponents less `shift`, off by 2^-24 of it: from 2^24 on they would have lost their last bit, and
// are not a number (a row of weight 0 has the shift inf, which makes them 0).
__device__ inline void finish_row(const Ce& c, int i, int64_t r, float z, float m, float others, float* row_loss,
                                  float* each) {
  const float mine = exp2_of(z - m), sum = others + mine;
  const float l = mine == 1.f ? log1pf(others) : (m - z) * kLn2 + logf(sum);
  const float coef = at<float>(c.saved, c.at.coef)[i];
  const float shift = m + log2f(sum) - log2f(coef);
  at<float>(c.saved, c.at.shift)[i] = coef > 0.f && !(fabsf(shift) < 0x1p24f) ? NAN : shift;
  at<float>(c.saved, c.at.own)[i] = -coef * (others / sum);
  each[i] = l;
  if (row_loss) row_loss[r] = l;
}

// What bf16 cuts off a row's own dz, that of its target and by far its largest: the products take the value rounded,
// and the rest is multiplied afterwards, so that dE of the targets is off by its own rounding and little else
// (gradients of 4,096 rows, 128,000 x 2,048: off by 0.24% of their norm without, 0.17% with, as with a dz in
// float32). A wave has the sums of NI blocks of 32 items and a list in LDS of the rows whose target is one of them:
// row * 128 + the place of the item. What it costs where targets follow their popularity, and few waves have many
// rows: the sweep of 5,120 rows, 100,000 x 64 163 -> 183 us, of 14,336, 876,000 x 128 5,192 -> 5,243; dE of 64,000 x
// 2,048 942 -> 994.
constexpr int kRestList = 1536;
template <int DP> constexpr int kRestRows = DP <= 128 ? 64 : 32;  // that are multiplied at a time
template <int DP> constexpr int kRests = kRestRows<DP> * Tile<__bf16, DP>::kRowB + 512;  // bytes of LDS that takes

// Lists rows from `next` on, up to `last`, as long as there is room for all that are looked at together, and returns
// their number. next: the first row that was not looked at. place(target): of the item among the wave's, or -1.
template <typename F>
__device__ inline int list_rests(const Ce& c, int64_t& next, int64_t last, uint32_t list, int lane, F place) {
  typedef int s32x4 __attribute__((ext_vector_type(4)));
  constexpr int kAtOnce = 4;
  const int32_t* targets = at<int32_t>(c.saved, c.at.target);
  int n = 0;
  for (; next < last && n <= kRestList - kAtOnce * 256; next += kAtOnce * 256) {
    s32x4 t[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t row = next + u * 256 + lane * 4;
      t[u] = s32x4{-1, -1, -1, -1};
      if (row < last) t[u] = *(const s32x4*)(targets + row);  // (next is a multiple of 4, and the array's end of 64)
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = next + u * 256 + lane * 4 + i;
        const int item = place(t[u][i]);
        const bool hit = row < last && item >= 0;
        const uint64_t m = __ballot(hit);
        if (m == 0) continue;
        if (hit)
          *(CUTBCE_LDS uint32_t*)(size_t)(list + (n + __popcll(m & (((uint64_t)1 << lane) - 1))) * 4) =
              (uint32_t)row * 128 + (uint32_t)item;
        n += __popcll(m);
      }
  }
  return n;
}

// Has add(d, features, items) multiply a list of n > 0 rows, sixteen at a time: operands of 32 features, block d of the
// rows' `cols` columns from H on (D apart), and of the blocks of items, `mine` being the lane's place in them. `lds`:
// kRests bytes of the wave's own. EARLY: how many times kRestRows rows are on their way (128 features, 876,000 items,
// the tile of the most popular ones: 240 us with one, 100 with two).
template <int DP, int NI, int EARLY, typename F>
__device__ inline void multiply_rests(const Ce& c, const __bf16* H, int cols, uint32_t list, int n, int mine,
                                      uint32_t lds, int lane, F add) {
  using Ti = Tile<__bf16, DP>;
  static_assert(NI <= 4, "");
  constexpr int kRows = kRestRows<DP>, kLoads = kRows * Ti::kCPR / 64, kStep = 64 / Ti::kCPR, NDB = Ti::kNDB;
  static_assert(kRests<DP> % Ti::kRowB == 0, "");
  const uint32_t rests = lds + kRows * Ti::kRowB;
  const float* own = at<float>(c.saved, c.at.own);
  const int h = lane / 32, r = lane / Ti::kCPR;
  auto apart = []() {  // what other lanes wrote is read, and what they read is written, in this order
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  // The rows of entries k, k + 1, ... (behind the last its row again, times 0; features past cols are not used), and
  // what was cut off each: item << 16 | rest in bf16, an entry a lane.
  u32x4 x[EARLY][kLoads];
  float cut[EARLY];
  uint32_t who[EARLY];
  auto load = [&](int a, int k) {
    auto entry = [&](int e) { return *(CUTBCE_LDS const uint32_t*)(size_t)(list + (e < n ? e : n - 1) * 4); };
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int chunk = (lane % Ti::kCPR) ^ Ti::swz(r) ^ Ti::swz(q * kStep % 32);
      const int64_t row = entry(k + r + q * kStep) >> 7;
      x[a][q] = *(const u32x4*)(H + row * c.D + (chunk * 8 < cols ? chunk * 8 : 0));
    }
    const uint32_t e = entry(k + lane);
    who[a] = e << 25 >> 9, cut[a] = own[e >> 7];
  };
  auto turn = [&](int a, int k) {
    apart();
#pragma unroll
    for (int q = 0; q < kLoads; ++q) *(CUTBCE_LDS u32x4*)(size_t)(lds + q * 1024 + lane * 16) = x[a][q];
    const __bf16 rest = (__bf16)(k + lane < n ? cut[a] - (float)(__bf16)cut[a] : 0.f);
    *(CUTBCE_LDS uint32_t*)(size_t)(rests + lane * 4) = who[a] | __builtin_bit_cast(uint16_t, rest);
    apart();
    load(a, k + EARLY * kRows);
#pragma unroll
    for (int g = 0; g < kRows / 16; ++g) {
      if (k + 16 * g >= n) break;
      u32x4 items[NI];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4 y = lds16(rests + (16 * g + 8 * j + 4 * h) * 4);
#pragma unroll
        for (int b = 0; b < NI; ++b) {
          uint32_t z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = (int)(y[i] >> 16) == b * 32 + mine ? y[i] : 0;
          items[b][2 * j] = __builtin_amdgcn_perm(z[1], z[0], 0x05040100u);  // (the low halves together)
          items[b][2 * j + 1] = __builtin_amdgcn_perm(z[3], z[2], 0x05040100u);
        }
      }
      const uint32_t base = Mma<__bf16>::base_t<DP>(lds + g / 2 * 32 * Ti::kRowB, lane);
#pragma unroll
      for (int d = 0; d < NDB; ++d) add(d, Mma<__bf16>::load_t<DP>(g % 2 * NDB + d, base), items);
    }
  };
  apart();
#pragma unroll
  for (int a = 0; a < EARLY; ++a) load(a, a * kRows);
  for (int k = 0; k < n; k += EARLY * kRows)
#pragma unroll
    for (int a = 0; a < EARLY; ++a)
      if (!a || k + a * kRows < n) turn(a, k + a * kRows);
  apart();
}

}  // namespace

}  // namespace cutbce
