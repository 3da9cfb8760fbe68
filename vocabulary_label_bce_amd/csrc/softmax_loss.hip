// Softmax cross entropy over a whole vocabulary, without keeping the logits.
//
//   z = scale H E^T,  lse_r = log sum_v exp z_rv,  l_r = lse_r - z_rt,  loss = sum w_r l_r / W
//   dz_rv = w_r / W (p_rv - [v = t_r]),  p = exp(z - lse),  dH = scale dz E,  dE = scale dz^T H
//
// Rows without a target are left out first (k_ce_rows), the others' H is copied together (k_ce_gather). Exponents are in
// base 2, c = |scale| log2 e times the products; a negative scale turns H's signs. A row's target is left out of the
// sums and products and joined in at the end: 1 - p_t is the others' share of the sum, and is exact to rounding where
// p_t is near 1, as a row's loss log(1 + others / e_t) is.
//
// The path of this file, for every size: the sums by one product kernel whose tiles are reduced where they are formed
// (k_ce_sums); the gradients in pieces of the vocabulary, for each of which dz is formed again, kept in 16 (32) bits and
// multiplied with E and with H (k_ce_dz, k_ce_dh, k_ce_de).
#include "softmax.h"

namespace cutbce {

namespace {

// ---------------------------------------------------------------------------------------------------------
// Rows: which have a target, their weights' sum, and their H together.
// ---------------------------------------------------------------------------------------------------------

// One workgroup; a wave has a range of rows and goes through it twice, counting first.
template <typename I>
__global__ __launch_bounds__(1024) void k_ce_rows(Ce c, const I* __restrict__ targets,
                                                  const float* __restrict__ weight) {
  __shared__ int count[16];
  __shared__ double sum[16];
  const int wave = uni(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int64_t share = up(cdiv(c.R, 16), 64), r0 = wave * share, r1 = r0 + share < c.R ? r0 + share : c.R;
  int n = 0;
  double w = 0;
#pragma unroll 4
  for (int64_t r = r0 + lane; r < r1; r += 64) {
    const int64_t t = targets[r];
    const bool in = t >= 0 && t < c.V;
    n += in;
    w += in ? (weight ? (double)weight[r] : 1.0) : 0.0;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64), w += __shfl_xor(w, o, 64);
  if (lane == 0) count[wave] = n, sum[wave] = w;
  __syncthreads();
  int from = 0, total = 0;
  double W = 0;
  for (int i = 0; i < 16; ++i) {
    if (i < wave) from += count[i];
    total += count[i];
    W += sum[i];
  }
  if (threadIdx.x == 0) *at<CeHead>(c.saved, c.at.head) = {total, (float)W};
  const double f = W > 0 ? 1.0 / W : (W == 0 ? 0.0 : W);  // (NaN stays)
  int32_t *rows = at<int32_t>(c.saved, c.at.rows), *place = at<int32_t>(c.saved, c.at.place),
          *target = at<int32_t>(c.saved, c.at.target);
  float* coef = at<float>(c.saved, c.at.coef);
  for (int64_t b = r0; b < r1; b += 64) {
    const int64_t r = b + lane;
    const int64_t t = r < r1 ? (int64_t)targets[r] : -1;
    const bool in = t >= 0 && t < c.V;
    const uint64_t m = __ballot(in);
    const int i = from + __popcll(m & (((uint64_t)1 << lane) - 1));
    if (in) {
      rows[i] = (int32_t)r;
      target[i] = (int32_t)t;
      coef[i] = (float)((weight ? (double)weight[r] : 1.0) * f);
    }
    if (r < r1) place[r] = in ? i : -1;
    from += __popcll(m);
  }
}

// A wave has a row: its copy, and c times its product with its target's item.
template <typename T>
__global__ __launch_bounds__(256) void k_ce_gather(Ce c, const T* __restrict__ H, float* __restrict__ zt) {
  const int i = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
  if (i >= at<CeHead>(c.saved, c.at.head)->n) return;
  const T* from = H + (int64_t)at<int32_t>(c.saved, c.at.rows)[i] * c.D;
  const T* item = (const T*)c.E + (int64_t)at<int32_t>(c.saved, c.at.target)[i] * c.D;
  T* to = at<T>(c.saved, c.at.hc) + (int64_t)i * c.D;
  const bool none = !(fabsf(c.scale) * kLog2e > 0.f);
  float s = 0.f;
  constexpr int N = Vec<T>::N;
  for (int d = lane * N; d < c.D; d += 64 * N) {
    float x[N], y[N];
    load_vec(from + d, x);
    load_vec(item + d, y);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j] = none ? 0.f : (c.scale < 0.f ? -x[j] : x[j]);
      s += x[j] * y[j];
    }
    store_vec(to + d, x);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if (lane == 0) zt[i] = s * base2(c.scale);
}

// ---------------------------------------------------------------------------------------------------------
// Products. A workgroup forms a tile of BM x BN results from stages of kStageK features (128 bytes) of both sides in
// LDS, two stages in turn: the loads of one are on their way while the other is multiplied.
// A side is read by rows (the features next to each other) or transposed (the results' index next to each other).
// ---------------------------------------------------------------------------------------------------------
template <typename T> constexpr int kStageK = 128 / sizeof(T);

template <typename T, int ROWS, bool TRANS, int NL> struct Side;

template <typename T, int ROWS, int NL> struct Side<T, ROWS, false, NL> {
  static constexpr int K = kStageK<T>, kBytes = ROWS * 128;
  using Ld = Dma<T, K, ROWS, NL>;
  Ld ld;
  int64_t stride;
  __device__ inline void init(int64_t s) { stride = s, ld.init(threadIdx.x, s); }
  // rows from `row` of `rows`, features from `k` of `left`
  __device__ inline void load(const T* base, int64_t row, int64_t rows, int64_t k, int64_t left, uint32_t dst) const {
    const int dh = (int)clamp64(left - k, 0, K);
    const u32x4 r = ld.range(base + row * stride + k, dh > 0 ? rows - row : 0, stride, dh);
#pragma unroll
    for (int q = 0; q < Ld::kRounds; ++q) ld.round(q, r, dh, dst);
  }
  __device__ static inline u32x4 op(uint32_t at, int block, int t, int lane) {
    return load_row(base_row<T, K>(at, lane) + block * 32 * 128, t);
  }
};

template <typename T, int ROWS, int NL> struct Side<T, ROWS, true, NL> {
  static constexpr int K = kStageK<T>, kSub = K * Tile<T, 128>::kRowB, kBytes = ROWS / 128 * kSub;
  using Ld = Dma<T, 128, K, NL>;
  Ld ld;
  int64_t stride;
  __device__ inline void init(int64_t s) { stride = s, ld.init(threadIdx.x, s); }
  __device__ inline void load(const T* base, int64_t row, int64_t rows, int64_t k, int64_t left, uint32_t dst) const {
#pragma unroll
    for (int b = 0; b < ROWS / 128; ++b) {
      const int dh = (int)clamp64(rows - row - b * 128, 0, 128);
      const u32x4 r = ld.range(base + k * stride + row + b * 128, dh > 0 ? left - k : 0, stride, dh);
#pragma unroll
      for (int q = 0; q < Ld::kRounds; ++q) ld.round(q, r, dh, dst + b * kSub);
    }
  }
  __device__ static inline u32x4 op(uint32_t at, int block, int t, int lane) {
    const uint32_t base = Mma<T>::template base_t<128>(at + block / 4 * kSub, lane);
    if constexpr (sizeof(T) == 2) {
      return __builtin_bit_cast(u32x4, Mma<T>::template load_t<128>(t * 4 + block % 4, base));
    } else {
      f32x4 x;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = Mma<T>::template load_t<128>((4 * t + j) * 4 + block % 4, base);
      return __builtin_bit_cast(u32x4, x);
    }
  }
};

template <typename T_, int WM_, int WN_, int TM_, int TN_, bool TA, bool TB> struct Product {
  using T = T_;
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
  static constexpr int NL = 64 * WM * WN, BM = WM * TM * 32, BN = WN * TN * 32, K = kStageK<T>;
  using A = Side<T, BM, TA, NL>;
  using B = Side<T, BN, TB, NL>;
  static constexpr int kStage = A::kBytes + B::kBytes, kLds = 2 * kStage;
  A a;
  B b;
  uint32_t lds0;
  int wave, lane, wm, wn;
  f32x16 acc[TM][TN];

  __device__ inline void init(char* lds, int64_t sa, int64_t sb) {
    lds0 = uni((uint32_t)(size_t)(CUTBCE_LDS char*)lds);
    wave = uni(threadIdx.x / 64), lane = threadIdx.x % 64;
    wm = wave % WM, wn = wave / WM;
    a.init(sa), b.init(sb);
    clear();
  }
  __device__ inline void clear() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};
  }
  __device__ inline uint32_t stage(int s) const { return lds0 + (s & 1) * kStage; }
  __device__ inline uint32_t wave_dst(int s) const { return stage(s) + wave * 1024; }
  // (the first load's wave kilobyte; every round of a side covers NL * 16 bytes)
  __device__ inline void multiply(int s) {
    const uint32_t pa = stage(s), pb = pa + A::kBytes;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      u32x4 x[TM], y[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) x[i] = A::op(pa, wm * TM + i, t, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) y[j] = B::op(pb, wn * TN + j, t, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = Mma<T>::mma(x[i], y[j], acc[i][j]);
    }
  }
};

// The sums: results are items x rows, so that a lane has one row's.
template <typename T> struct Sizes {
  using Sums = Product<T, 2, 2, 2, 2, false, false>;
  using Dh = Product<T, 2, 2, 2, 2, false, true>;
  using De = Product<T, 2, 2, 2, 2, true, true>;
};

// Units of work: tiles of rows x shares of the vocabulary, the shares' number from that of the tiles. Neighbouring
// units, which read the same items, go to workgroups of one XCD (every eighth).
struct Units {
  int tiles, shares;
};
__device__ inline Units units_of(int n, int64_t V, int bm, int bn, int grid) {
  Units u;
  u.tiles = (n + bn - 1) / bn;
  const int64_t steps = (V + bm - 1) / bm;
  int64_t s = u.tiles ? grid / u.tiles : 1;
  s = s > steps ? steps : s;
  u.shares = s < 1 ? 1 : (int)s;
  return u;
}
constexpr int kCeGrid = 512;  // workgroups of the sums: two a CU

template <typename P>
__global__ __launch_bounds__(P::NL, 2) void k_ce_sums(Ce c, float2* __restrict__ part) {
  using T = typename P::T;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const Units units = units_of(n, c.V, P::BM, P::BN, gridDim.x);
  const int total = units.tiles * units.shares, per = (total + 7) / 8;
  P p;
  p.init(lds, c.D, c.D);
  const T *E = (const T*)c.E, *H = at<T>(c.saved, c.at.hc);
  const float cc = base2(c.scale);
  const int32_t* targets = at<int32_t>(c.saved, c.at.target);
  const int64_t steps = (c.V + P::BM - 1) / P::BM;
  const int nk = (c.D + P::K - 1) / P::K, h = p.lane / 32;
  for (int k = blockIdx.x / 8; k < per; k += gridDim.x / 8) {
    const int u = (blockIdx.x % 8) * per + k;
    if (u >= total) break;
    const int tile = u % units.tiles, share = u / units.tiles;
    const int64_t v0 = steps * share / units.shares, v1 = steps * (share + 1) / units.shares;
    const int64_t row0 = (int64_t)tile * P::BN;
    float m[P::TN], s[P::TN];
    int64_t target[P::TN];
#pragma unroll
    for (int j = 0; j < P::TN; ++j) {
      const int64_t i = row0 + (p.wn * P::TN + j) * 32 + p.lane % 32;
      m[j] = -INFINITY, s[j] = 0.f;
      target[j] = i < n ? targets[i] : -1;
    }
    const int64_t all = (v1 - v0) * nk;
    auto fetch = [&](int64_t x) {
      if (x >= all) return;
      const int64_t v = (v0 + x / nk) * P::BM, kk = x % nk * P::K;
      const uint32_t dst = p.wave_dst((int)(x & 1));
      p.a.load(E, v, c.V, kk, c.D, dst);
      p.b.load(H, row0, n, kk, c.D, dst + P::A::kBytes);
    };
    wait_and_sync<>();  // (the unit before is done with both stages)
    fetch(0);
    for (int64_t x = 0; x < all; ++x) {
      wait_and_sync<>();
      fetch(x + 1);
      p.multiply((int)(x & 1));
      if (x % nk != nk - 1) continue;
      const int64_t v = (v0 + x / nk) * P::BM + p.wm * P::TM * 32;
#pragma unroll
      for (int j = 0; j < P::TN; ++j) {
        if (__any((target[j] >= v && target[j] < v + P::TM * 32) || v + P::TM * 32 > c.V)) {
#pragma unroll
          for (int i = 0; i < P::TM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int64_t item = v + i * 32 + acc_row(e, h);
              if (item == target[j] || item >= c.V) p.acc[i][j][e] = -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < P::TM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, p.acc[i][j][e]);
        const float next = fmaxf(m[j], top * cc), base = next == -INFINITY ? 0.f : next;
        s[j] *= exp2_of(m[j] - base);
        m[j] = next;
#pragma unroll
        for (int i = 0; i < P::TM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[j] += exp2_of(__builtin_fmaf(p.acc[i][j][e], cc, -base));
      }
      p.clear();
    }
    const int slots = units.shares * P::WM, slot = share * P::WM + p.wm;
#pragma unroll
    for (int j = 0; j < P::TN; ++j) {
      const int64_t i = row0 + (p.wn * P::TN + j) * 32 + p.lane % 32;
      const float om = other_half(m[j]), os = other_half(s[j]);
      const float top = fmaxf(m[j], om), base = top == -INFINITY ? 0.f : top;
      if (i < n && h == 0)
        part[i * slots + slot] = make_float2(top, s[j] * exp2_of(m[j] - base) + os * exp2_of(om - base));
    }
  }
}

// A wave has a row of the batch: joins its shares' sums.
struct JoinHow {
  int bm, bn, grid, slots;  // of the kernel that left the sums; slots for each share
};
__global__ __launch_bounds__(256) void k_ce_join(Ce c, JoinHow how, const float2* __restrict__ part,
                                                 const float* __restrict__ zt, float* __restrict__ row_loss,
                                                 float* __restrict__ each) {
  const int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int lane = threadIdx.x % 64;
  if (r >= c.R) return;
  const int i = at<int32_t>(c.saved, c.at.place)[r];
  if (i < 0) {
    if (lane == 0 && row_loss) row_loss[r] = 0.f;
    return;
  }
  const Units u = units_of(at<CeHead>(c.saved, c.at.head)->n, c.V, how.bm, how.bn, how.grid);
  const int slots = u.shares * how.slots;
  const float z = zt[i];
  float m = z;
  for (int k = lane; k < slots; k += 64) m = fmaxf(m, part[(int64_t)i * slots + k].x);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  float others = 0.f;
  for (int k = lane; k < slots; k += 64) {
    const float2 x = part[(int64_t)i * slots + k];
    others += x.y == 0.f ? 0.f : x.y * exp2_of(x.x - m);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) others += __shfl_xor(others, o, 64);
  if (lane) return;
  const float mine = exp2_of(z - m), sum = others + mine;
  const float l = mine == 1.f ? log1pf(others) : (m - z) * kLn2 + logf(sum);
  at<float>(c.saved, c.at.lse)[i] = m + log2f(sum);
  at<float>(c.saved, c.at.rest)[i] = others / sum;
  each[i] = l;
  if (row_loss) row_loss[r] = l;
}

__global__ __launch_bounds__(1024) void k_ce_loss(Ce c, const float* __restrict__ each, float* __restrict__ loss) {
  __shared__ double part[16];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const float* coef = at<float>(c.saved, c.at.coef);
  double s = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += 1024) s += (double)coef[i] * (double)each[i];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0;
    for (int i = 0; i < 16; ++i) s += part[i];
    *loss = (float)s;
  }
}

// ---------------------------------------------------------------------------------------------------------
// Gradients, a piece of the vocabulary at a time: items v0 .. v0 + width - 1 (width a multiple of 256).
// ---------------------------------------------------------------------------------------------------------

// dz of the piece, [n][width] (zeros for items behind the vocabulary's end). In 16 bits the items of each 16 stand in the
// order 0-3, 8-11, 4-7, 12-15: a lane's eight results are next to each other, and are the operand of the product with E
// in the order in which the transposed reads of E give their items.
__host__ __device__ constexpr inline int item_at(int place) {  // of 16 bits
  return (place & ~12) | (place & 4) << 1 | (place & 8) >> 1;
}
template <typename P>
__global__ __launch_bounds__(P::NL, 2) void k_ce_dz(Ce c, int64_t v0, int64_t width, typename P::T* __restrict__ dz) {
  using T = typename P::T;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int tiles = (int)(width / P::BM);  // of items; neighbours read the same rows
  const int64_t row0 = (int64_t)(blockIdx.x / tiles) * P::BN, v = v0 + (int64_t)(blockIdx.x % tiles) * P::BM;
  if (row0 >= n) return;
  P p;
  p.init(lds, c.D, c.D);
  const T *E = (const T*)c.E, *H = at<T>(c.saved, c.at.hc);
  const int nk = (c.D + P::K - 1) / P::K, h = p.lane / 32;
  auto fetch = [&](int x) {
    if (x >= nk) return;
    p.a.load(E, v, c.V, x * P::K, c.D, p.wave_dst(x));
    p.b.load(H, row0, n, x * P::K, c.D, p.wave_dst(x) + P::A::kBytes);
  };
  fetch(0);
  for (int x = 0; x < nk; ++x) {
    wait_and_sync<>();
    fetch(x + 1);
    p.multiply(x);
  }
  const float cc = base2(c.scale);
#pragma unroll
  for (int j = 0; j < P::TN; ++j) {
    const int64_t i = row0 + (p.wn * P::TN + j) * 32 + p.lane % 32;
    if (i >= n) continue;
    const float lse = at<float>(c.saved, c.at.lse)[i], coef = at<float>(c.saved, c.at.coef)[i];
    const float mine = -coef * at<float>(c.saved, c.at.rest)[i];
    const int64_t target = at<int32_t>(c.saved, c.at.target)[i];
#pragma unroll
    for (int b = 0; b < P::TM; ++b) {
      const int64_t first = v + (p.wm * P::TM + b) * 32;
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t item = first + acc_row(e, h);
        x[e] = coef * exp2_of(__builtin_fmaf(p.acc[b][j][e], cc, -lse));
        x[e] = item == target ? mine : (item < c.V ? x[e] : 0.f);
      }
      T* to = dz + i * width + (first - v0);
      if constexpr (sizeof(T) == 2) {
        store_vec(to + 8 * h, x);
        store_vec(to + 16 + 8 * h, x + 8);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) store_vec(to + 8 * k + 4 * h, x + 4 * k);
      }
    }
  }
}

// sums[part] (+)= dz E over the part's items: rows x features.
template <typename P>
__global__ __launch_bounds__(P::NL, 2) void k_ce_dh(Ce c, int64_t v0, int64_t width, int parts, int first,
                                                    const typename P::T* __restrict__ dz, float* __restrict__ sums) {
  using T = typename P::T;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int cols = (c.D + P::BN - 1) / P::BN;
  const int part = blockIdx.x % parts, tile = blockIdx.x / parts;
  const int64_t row0 = (int64_t)(tile / cols) * P::BM, d0 = (int64_t)(tile % cols) * P::BN;
  if (row0 >= n) return;
  P p;
  p.init(lds, width, c.D);
  const int64_t left = c.V - v0 < width ? c.V - v0 : width, steps = (left + P::K - 1) / P::K;
  const int64_t x0 = steps * part / parts, x1 = steps * (part + 1) / parts;
  const T* E = (const T*)c.E + v0 * c.D;
  auto fetch = [&](int64_t x) {
    if (x >= x1) return;
    const uint32_t dst = p.wave_dst((int)(x & 1));
    p.a.load(dz, row0, n, x * P::K, width, dst);
    p.b.load(E, d0, c.D, x * P::K, left, dst + P::A::kBytes);
  };
  fetch(x0);
  for (int64_t x = x0; x < x1; ++x) {
    wait_and_sync<>();
    fetch(x + 1);
    p.multiply((int)(x & 1));
  }
  float* to = sums + (int64_t)part * c.R * c.D;
  const int h = p.lane / 32;
#pragma unroll
  for (int i = 0; i < P::TM; ++i)
#pragma unroll
    for (int j = 0; j < P::TN; ++j) {
      const int64_t d = d0 + (p.wn * P::TN + j) * 32 + p.lane % 32;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t row = row0 + (p.wm * P::TM + i) * 32 + acc_row(e, h);
        if (row < n && d < c.D) {
          float* x = to + row * c.D + d;
          *x = first ? p.acc[i][j][e] : *x + p.acc[i][j][e];
        }
      }
    }
}

// dE of the piece: items x features, over all rows; or a part of the rows, to be joined.
template <typename P, bool PART>
__global__ __launch_bounds__(P::NL, 2) void k_ce_de(Ce c, int64_t v0, int64_t width, int parts,
                                                    const typename P::T* __restrict__ dz, const float* __restrict__ grad,
                                                    typename P::T* __restrict__ dE, float* __restrict__ sums) {
  using T = typename P::T;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int cols = (c.D + P::BN - 1) / P::BN;
  const int part = PART ? blockIdx.x % parts : 0, tile = PART ? blockIdx.x / parts : blockIdx.x;
  const int64_t u0 = (int64_t)(tile / cols) * P::BM, d0 = (int64_t)(tile % cols) * P::BN;
  if (v0 + u0 >= c.V) return;
  P p;
  p.init(lds, width, c.D);
  const T* H = at<T>(c.saved, c.at.hc);
  const int64_t steps = (n + P::K - 1) / P::K;
  const int64_t x0 = PART ? steps * part / parts : 0, x1 = PART ? steps * (part + 1) / parts : steps;
  auto fetch = [&](int64_t x) {
    if (x >= x1) return;
    const uint32_t dst = p.wave_dst((int)(x & 1));
    p.a.load(dz, u0, width, x * P::K, n, dst);
    p.b.load(H, d0, c.D, x * P::K, n, dst + P::A::kBytes);
  };
  fetch(x0);
  for (int64_t x = x0; x < x1; ++x) {
    wait_and_sync<>();
    fetch(x + 1);
    p.multiply((int)(x & 1));
  }
  const float f = PART ? 1.f : *grad * fabsf(c.scale);
  const int h = p.lane / 32;
#pragma unroll
  for (int i = 0; i < P::TM; ++i)
#pragma unroll
    for (int j = 0; j < P::TN; ++j) {
      const int64_t d = d0 + (p.wn * P::TN + j) * 32 + p.lane % 32;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        int64_t u = u0 + (p.wm * P::TM + i) * 32 + acc_row(e, h);
        if (sizeof(T) == 2) u = item_at((int)u);
        if (v0 + u < c.V && d < c.D) {
          if constexpr (PART) sums[((int64_t)part * width + u) * c.D + d] = p.acc[i][j][e];
          else dE[(v0 + u) * c.D + d] = from_f32<T>(p.acc[i][j][e] * f);
        }
      }
    }
}

// dE of a piece from its parts' sums: four features a lane.
template <typename T>
__global__ __launch_bounds__(256) void k_ce_de_join(Ce c, int64_t v0, int64_t width, int parts,
                                                    const float* __restrict__ sums, const float* __restrict__ grad,
                                                    T* __restrict__ dE) {
  const int64_t left = c.V - v0 < width ? c.V - v0 : width;
  const int64_t x = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (x >= left * c.D) return;
  const float f = *grad * fabsf(c.scale);
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < parts; ++k) s += *(const f32x4*)(sums + (int64_t)k * width * c.D + x);
  typedef T V4 __attribute__((ext_vector_type(4)));
  V4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = from_f32<T>(s[j] * f);
  *(V4*)(dE + v0 * c.D + x) = y;
}

// dH of all rows, zeros for those without a target: four features a lane, the sum of the parts'.
template <typename T>
__global__ __launch_bounds__(256) void k_ce_dh_join(Ce c, int parts, const float* __restrict__ sums,
                                                    const float* __restrict__ grad, T* __restrict__ dH) {
  const int64_t x = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (x >= c.R * c.D) return;
  const int64_t r = x / c.D;
  const int i = at<int32_t>(c.saved, c.at.place)[r];
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (i >= 0) {
    const int64_t from = (int64_t)i * c.D + (x - r * c.D);
    for (int k = 0; k < parts; ++k) s += *(const f32x4*)(sums + (int64_t)k * c.R * c.D + from);
    s *= *grad * c.scale;
  }
  typedef T V4 __attribute__((ext_vector_type(4)));
  V4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = from_f32<T>(s[j]);
  *(V4*)(dH + x) = y;
}

// ---------------------------------------------------------------------------------------------------------
// Sizes and launches.
// ---------------------------------------------------------------------------------------------------------
struct Plan {
  int64_t width;           // items of a piece
  int dh_parts, de_parts;
  size_t dz, dh, de, bytes;  // offsets in the workspace
};
int64_t clamp_parts(int64_t tiles, int64_t steps, int64_t most) {
  int64_t parts = tiles < 512 ? 512 / (tiles ? tiles : 1) : 1;  // two workgroups a CU
  if (parts > steps / 4) parts = steps / 4;                     // each at least four stages
  if (parts > most) parts = most;
  return parts < 1 ? 1 : parts;
}
template <typename T> Plan plan_of(int64_t R, int64_t V, int D) {
  using S = Sizes<T>;
  if (R < 1) R = 1;
  Plan p;
  // a piece's dz takes up to 256 MB, the size of the memory-side cache
  int64_t width = ((int64_t)256 << 20) / (R * (int64_t)sizeof(T)) / 256 * 256;
  if (width < 256) width = 256;
  if (width > up(V, 256)) width = up(V, 256);
  if (width > (int64_t)1 << 22) width = (int64_t)1 << 22;  // (offsets inside a stage are 32-bit)
  p.width = width;
  p.dh_parts = (int)clamp_parts(cdiv(R, S::Dh::BM) * cdiv(D, S::Dh::BN), width / kStageK<T>,
                                ((int64_t)256 << 20) / (R * D * 4) + 1);
  p.de_parts = (int)clamp_parts(width / S::De::BM * cdiv(D, S::De::BN), cdiv(R, kStageK<T>), 64);
  size_t b = 0;
  p.dz = b, b += up(R * width * (int64_t)sizeof(T), 256);
  p.dh = b, b += up((int64_t)p.dh_parts * R * D * 4, 256);
  p.de = b, b += p.de_parts > 1 ? up((int64_t)p.de_parts * width * D * 4, 256) : 0;
  p.bytes = b;
  return p;
}

struct ForwardPlan {
  size_t zt, each, part, bytes;
};
template <typename T> ForwardPlan forward_plan(int64_t R, int D, bool grad) {
  using P = typename Sizes<T>::Sums;
  ForwardPlan f;
  size_t b = 0;
  f.zt = b, b += up(R * 4, 256);
  f.each = b, b += up(R * 4, 256);
  if (ce_swept(D, sizeof(T) == 2)) {
    f.part = b, b += ce_rows_bytes(R, D, grad);
    f.bytes = b;
    return f;
  }
  // shares x tiles of rows are at most the grid, or one share each
  const int64_t tiles = cdiv(R, P::BN);
  f.part = b, b += up((tiles > kCeGrid ? tiles : kCeGrid) * P::BN * P::WM * 8, 256);
  f.bytes = b;
  return f;
}

template <typename T>
hipError_t forward_t(const Ce& c, int id_bytes, const T* H, const void* targets, const float* weight, bool grad,
                     float* loss, float* row_loss, hipStream_t st) {
  using P = typename Sizes<T>::Sums;
  const ForwardPlan f = forward_plan<T>(c.R, c.D, grad);
  float *zt = (float*)(c.ws + f.zt), *each = (float*)(c.ws + f.each);
  float2* part = (float2*)(c.ws + f.part);
  if (id_bytes == 4) k_ce_rows<int32_t><<<1, 1024, 0, st>>>(c, (const int32_t*)targets, weight);
  else k_ce_rows<int64_t><<<1, 1024, 0, st>>>(c, (const int64_t*)targets, weight);
  if (c.R) k_ce_gather<T><<<(unsigned)cdiv(c.R, 4), 256, 0, st>>>(c, H, zt);
  if (ce_swept(c.D, c.dtype)) {
    const hipError_t e = c.R ? launch_ce_rows(c, c.ws + f.part, grad, zt, row_loss, each, st) : hipSuccess;
    if (e != hipSuccess) return e;
  } else if (c.R) {
    const hipError_t e = allow_lds<k_ce_sums<P>>(P::kLds);
    if (e != hipSuccess) return e;
    k_ce_sums<P><<<kCeGrid, P::NL, P::kLds, st>>>(c, part);
    k_ce_join<<<(unsigned)cdiv(c.R, 4), 256, 0, st>>>(c, JoinHow{P::BM, P::BN, kCeGrid, P::WM}, part, zt, row_loss, each);
  }
  k_ce_loss<<<1, 1024, 0, st>>>(c, each, loss);
  return hipGetLastError();
}

template <typename T> hipError_t backward_t(const Ce& c, const float* grad, T* dH, T* dE, hipStream_t st) {
  using S = Sizes<T>;
  const Plan p = plan_of<T>(c.R, c.V, c.D);
  T* dz = (T*)(c.ws + p.dz);
  float *dh = (float*)(c.ws + p.dh), *de = (float*)(c.ws + p.de);
  hipError_t e = allow_lds<k_ce_dz<typename S::Sums>>(S::Sums::kLds);
  if (e == hipSuccess) e = allow_lds<k_ce_dh<typename S::Dh>>(S::Dh::kLds);
  if (e == hipSuccess) e = allow_lds<k_ce_de<typename S::De, false>>(S::De::kLds);
  if (e == hipSuccess) e = allow_lds<k_ce_de<typename S::De, true>>(S::De::kLds);
  if (e != hipSuccess) return e;
  for (int64_t v = 0; v < c.V; v += p.width) {
    if (c.R) k_ce_dz<typename S::Sums><<<(unsigned)(cdiv(c.R, S::Sums::BN) * (p.width / S::Sums::BM)), S::Sums::NL, S::Sums::kLds,
                                st>>>(c, v, p.width, dz);
    if (dH && c.R)
      k_ce_dh<typename S::Dh><<<(unsigned)(cdiv(c.R, S::Dh::BM) * cdiv(c.D, S::Dh::BN) * p.dh_parts), S::Dh::NL,
                                S::Dh::kLds, st>>>(c, v, p.width, p.dh_parts, v == 0, dz, dh);
    if (dE) {
      const unsigned tiles = (unsigned)(p.width / S::De::BM * cdiv(c.D, S::De::BN));
      if (p.de_parts > 1) {
        k_ce_de<typename S::De, true><<<tiles * p.de_parts, S::De::NL, S::De::kLds, st>>>(c, v, p.width, p.de_parts, dz,
                                                                                         grad, dE, de);
        k_ce_de_join<T><<<(unsigned)cdiv(p.width * c.D, 1024), 256, 0, st>>>(c, v, p.width, p.de_parts, de, grad, dE);
      } else {
        k_ce_de<typename S::De, false><<<tiles, S::De::NL, S::De::kLds, st>>>(c, v, p.width, 1, dz, grad, dE, de);
      }
    }
  }
  if (dH && c.R) k_ce_dh_join<T><<<(unsigned)cdiv(c.R * c.D, 1024), 256, 0, st>>>(c, p.dh_parts, dh, grad, dH);
  return hipGetLastError();
}

}  // namespace

CeSaved ce_saved(int64_t R, int64_t V, int D, int dtype) {
  CeSaved s;
  size_t b = 0;
  s.head = b, b += 256;
  size_t* each[] = {&s.rows, &s.place, &s.target, &s.lse, &s.rest, &s.coef};
  for (size_t* x : each) *x = b, b += up(R * 4, 256);
  s.hc = b, b += up(R * D * (dtype ? 2 : 4), 256);
  s.dh = b, b += ce_swept(D, dtype) ? up(R * D * 4, 256) : 0;
  s.bytes = b;
  return s;
}

size_t ce_forward_bytes(int64_t R, int64_t V, int D, int dtype, bool want_grad) {
  const size_t own = dtype ? forward_plan<__bf16>(R, D, want_grad).bytes : forward_plan<float>(R, D, want_grad).bytes;
  return own + (want_grad ? 0 : ce_saved(R, V, D, dtype).bytes);
}
size_t ce_backward_bytes(int64_t R, int64_t V, int D, int dtype) {
  if (ce_swept(D, dtype)) return ce_items_bytes(R, V, D);
  return dtype ? plan_of<__bf16>(R, V, D).bytes : plan_of<float>(R, V, D).bytes;
}

hipError_t launch_ce_forward(const Ce& c, int id_bytes, const void* H, const void* targets, const float* weight,
                             bool want_grad, float* loss, float* row_loss, hipStream_t st) {
  return c.dtype ? forward_t<__bf16>(c, id_bytes, (const __bf16*)H, targets, weight, want_grad, loss, row_loss, st)
                 : forward_t<float>(c, id_bytes, (const float*)H, targets, weight, want_grad, loss, row_loss, st);
}
hipError_t launch_ce_backward(const Ce& c, const float* grad, void* dH, void* dE, hipStream_t st) {
  if (ce_swept(c.D, c.dtype)) return launch_ce_items(c, c.ws, grad, dH, dE, st);
  return c.dtype ? backward_t<__bf16>(c, grad, (__bf16*)dH, (__bf16*)dE, st)
                 : backward_t<float>(c, grad, (float*)dH, (float*)dE, st);
}

}  // namespace cutbce
