// Softmax cross entropy over a whole vocabulary, without keeping the logits.
//
//   z = scale H E^T,  lse_r = log sum_v exp z_rv,  l_r = lse_r - z_rt,  loss = sum w_r l_r / W
//   dz_rv = w_r / W (p_rv - [v = t_r]),  p = exp(z - lse),  dH = scale dz E,  dE = scale dz^T H
//
// Rows without a target are left out first, the others' H is copied together (k_ce_rows). Exponents are in
// base 2, c = |scale| log2 e times the products; a negative scale turns H's signs. A row's target is left out of the
// sums and products and joined in at the end: 1 - p_t is the others' share of the sum, and is exact to rounding where
// p_t is near 1, as a row's loss log(1 + others / e_t) is.
//
// The path of this file, for float32 and for bf16 rows of more than 256 features: the sums by one product kernel
// whose tiles are reduced where they are formed (k_ce_sums); the gradients in pieces of the vocabulary, for each of
// which dz is formed again, kept in 16 (32) bits and multiplied with E and with H (k_ce_dz, k_ce_dh, k_ce_de). The
// matrix units bound it: 4,096 rows, 128,000 items of 2,048 features, bf16, 0.95 to 1.25 PFLOP/s in the four
// products, dH the most (a large product of the library: 1.30); 768 x 65,536 x 256 in float32 112 to 118 TFLOP/s
// (154) in each. 739 rows of 65,537 items take as long as 768 (six tiles), and the one item more a seventh turn of a
// few tiles: 3% in the sums, 5% in dz; in dE a third round of the chip for two tiles (231 us, so 276).
#include "softmax.h"

namespace cutbce {

namespace {

// ---------------------------------------------------------------------------------------------------------
// Rows: which have a target, their weights' sum, and their H together.
// ---------------------------------------------------------------------------------------------------------

// A workgroup has a range of rows, each wave one at a time: its place among the counted ones, its copy, and c times its
// product with its target's item. All of them count all targets first, which is what one of them would have to do
// before the others could start. Latency bounds it: 5.4 us for 32 rows of 64 (two launches: 6.6), 28 for 25,600 of
// 128 (25), most of it the count.
template <typename T, typename I>
__global__ __launch_bounds__(1024) void k_ce_rows(Ce c, const T* __restrict__ H, const I* __restrict__ targets,
                                                  const float* __restrict__ weight, float* __restrict__ zt) {
  __shared__ int count[16], early[16], list[1024], aims[1024];
  __shared__ double sum[16];
  const int wave = uni(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int64_t share = cdiv(c.R, gridDim.x), r0 = blockIdx.x * share, r1 = r0 + share < c.R ? r0 + share : c.R;
  int n = 0, before = 0;
  double w = 0;
#pragma unroll 4
  for (int64_t r = threadIdx.x; r < c.R; r += 1024) {
    const int64_t t = targets[r];
    const bool in = t >= 0 && t < c.V;
    n += in;
    before += in && r < r0;
    w += in ? (weight ? (double)weight[r] : 1.0) : 0.0;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1)
    n += __shfl_xor(n, o, 64), before += __shfl_xor(before, o, 64), w += __shfl_xor(w, o, 64);
  if (lane == 0) count[wave] = n, early[wave] = before, sum[wave] = w;
  __syncthreads();
  int from = 0, total = 0;
  double W = 0;
  for (int i = 0; i < 16; ++i) from += early[i], total += count[i], W += sum[i];
  if (blockIdx.x == 0 && threadIdx.x == 0) *at<CeHead>(c.saved, c.at.head) = {total, (float)W};
  const double f = W > 0 ? 1.0 / W : (W == 0 ? 0.0 : W);  // (NaN stays)
  const bool none = !(fabsf(c.scale) * kLog2e > 0.f);
  int32_t *rows = at<int32_t>(c.saved, c.at.rows), *place = at<int32_t>(c.saved, c.at.place),
          *target = at<int32_t>(c.saved, c.at.target);
  float* coef = at<float>(c.saved, c.at.coef);
  for (int64_t b = r0; b < r1; b += 1024) {
    const int64_t r = b + threadIdx.x;
    const int64_t t = r < r1 ? (int64_t)targets[r] : -1;
    const bool in = t >= 0 && t < c.V;
    const uint64_t m = __ballot(in);
    __syncthreads();  // (the last turn's lists are read, and the counts)
    if (lane == 0) count[wave] = __popcll(m);
    __syncthreads();
    int k = __popcll(m & (((uint64_t)1 << lane) - 1)), here = 0;
    for (int i = 0; i < 16; ++i) k += i < wave ? count[i] : 0, here += count[i];
    if (in) {
      rows[from + k] = (int32_t)r;
      target[from + k] = (int32_t)t;
      coef[from + k] = (float)((weight ? (double)weight[r] : 1.0) * f);
      list[k] = (int)(r - b), aims[k] = (int)t;
    }
    if (r < r1) place[r] = in ? from + k : -1;
    __syncthreads();
    for (int j = wave; j < here; j += 16) {
      const T* x_at = H + (b + list[j]) * c.D;
      const T* item = (const T*)c.E + (int64_t)aims[j] * c.D;
      T* to = at<T>(c.saved, c.at.hc) + (int64_t)(from + j) * c.D;
      float s = 0.f;
      constexpr int N = Vec<T>::N;
      for (int d = lane * N; d < c.D; d += 64 * N) {
        float x[N], y[N];
        load_vec(x_at + d, x);
        load_vec(item + d, y);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          x[q] = none ? 0.f : (c.scale < 0.f ? -x[q] : x[q]);
          s += x[q] * y[q];
        }
        store_vec(to + d, x);
      }
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
      if (lane == 0) zt[from + j] = s * base2(c.scale);
    }
    from += here;
  }
}

// ---------------------------------------------------------------------------------------------------------
// Products. A workgroup forms a tile of BM x BN results from stages of KB bytes of features (K of them) of both
// sides, in a ring of kRing stages in LDS. Turn s multiplies stage s; stage s + 1 has landed by then, so that its
// first operands are read while the last products of stage s run, and the stages behind it are on their way. Two
// waves a SIMD; the order of matrix instructions and reads is pinned, a step's operands being read behind the
// products of the step before. A side is read by rows (the features next to each other) or transposed (the results'
// index next to each other).
// --------------------------------------------------------------------------------------------------------- 1, 2 or 4
// loads of 16 bytes a lane, as load_lds16 does them one by one: from bytes voff[] of the buffer to LDS bytes dst, dst
// + STEP, ... (+ lane * 16). A stage's loads are what its turn waits for and its scalar work: one block with one wait
// for its operands (as load_lds16 has), and what does not change from stage to stage formed before (the products of
// 4,096 rows with 32,768 items of 2,048 features took a third longer with the ranges formed for each stage).
template <int N, int STEP> __device__ inline void load_lds16s(u32x4 buffer, const int* voff, uint32_t dst) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 1) {
    load_lds16(buffer, voff[0], dst);
  } else if constexpr (N == 2) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %4\n\ts_nop 1\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
                 :: "s"(uni(dst)), "v"(voff[0]), "v"(voff[1]), "s"(buffer), "n"(STEP) : "m0", "scc");
  } else {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 1\n\tbuffer_load_dwordx4 %2, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 1\n\tbuffer_load_dwordx4 %3, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 1\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 :: "s"(uni(dst)), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3]), "s"(buffer), "n"(STEP)
                 : "m0", "scc");
  }
}

template <typename T, int ROWS, bool TRANS, int NL, int KB> struct Side;

template <typename T, int ROWS, int NL, int KB> struct Side<T, ROWS, false, NL, KB> {
  static constexpr int K = KB / sizeof(T), kBytes = ROWS * KB;
  using Ld = Dma<T, K, ROWS, NL>;
  static_assert(Tile<T, K>::kRowB == KB && Ld::kLanes == NL, "");
  static constexpr int kLoads = Ld::kRounds;
  Ld ld;
  int64_t stride, step;  // of rows, and of stages
  const T* from;  // of the next stage
  int whole, left;  // bytes of a whole stage's range; features left
  int voff[kLoads];
  __device__ inline void init(int64_t s) {
    stride = s, step = K, ld.init(threadIdx.x, s);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) voff[q] = ld.offset(q, K);
  }
  __device__ inline void init_blocked(int64_t rows) { init(K), step = rows * K; }
  // stages from row `row` of `rows`, feature k of `end`, on
  __device__ inline void start(const T* base, int64_t row, int64_t rows, int64_t k, int64_t end) {
    const int64_t r = clamp64(rows - row, 0, ROWS);
    from = base + row * stride + k / K * step + k % K;
    whole = r > 0 ? (int)(((r - 1) * stride + K) * sizeof(T)) : 0;
    left = r > 0 && end > k ? (int)(end - k) : 0;
  }
  // loads the next stage: zeros past the last feature, nothing (but as many loads) behind the last stage
  __device__ inline void load(uint32_t dst) {
    if (__builtin_expect(left >= K, 1)) {
      load_lds16s<kLoads, NL * 16>(buffer_of(from, whole), voff, dst);
    } else {
      int v[kLoads];
#pragma unroll
      for (int q = 0; q < kLoads; ++q) v[q] = ld.offset(q, left);
      load_lds16s<kLoads, NL * 16>(buffer_of(from, left > 0 ? whole - (K - left) * (int)sizeof(T) : 0), v, dst);
    }
    from += step, left -= left > 0 ? (left < K ? left : K) : 0;
  }
  __device__ static inline u32x4 op(uint32_t at, int block, int t, int lane) {
    return load_row(base_row<T, K>(at, lane) + block * 32 * KB, t);
  }
};

template <typename T, int ROWS, int NL, int KB> struct Side<T, ROWS, true, NL, KB> {
  static constexpr int K = KB / sizeof(T), kSub = K * Tile<T, 128>::kRowB, kBytes = ROWS / 128 * kSub;
  using Ld = Dma<T, 128, K, NL>;
  static_assert(Ld::kLanes == NL && kSub == Ld::kRounds * NL * 16, "");
  static constexpr int kLoads = ROWS / 128 * Ld::kRounds;
  Ld ld;
  int64_t stride;
  const T* from;
  int cols, left;  // of the tile's results; features left
  int whole;       // blocked: bytes of a stage's range
  int voff[kLoads];
  __device__ inline void init(int64_t s) { stride = s, whole = 0, ld.init(threadIdx.x, s); }
  // Blocked: all results and features of a stage are there.
  __device__ inline void init_blocked(int64_t rows) {
    constexpr int C = KB / sizeof(T);  // of a block
    init(C);
    whole = (int)(((ROWS / C - 1) * rows + K) * KB);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int round = q % Ld::kRounds, row = threadIdx.x / Ld::Ti::kCPR + round * Ld::kStep;
      const int x = (ld.chunk ^ Ld::Ti::swz(round * Ld::kStep)) * 16 + q / Ld::kRounds * 128 * (int)sizeof(T);
      voff[q] = x / KB * (int)(rows * KB) + row * KB + x % KB;
    }
  }
  __device__ inline void start_blocked(const T* base, int64_t block, int64_t rows, int64_t k, int64_t end) {
    from = base + (block * rows + k) * stride;
    left = end > k ? (int)(end - k) : 0;
  }
  __device__ inline void start(const T* base, int64_t row, int64_t rows, int64_t k, int64_t end) {
    from = base + k * stride + row;
    cols = (int)clamp64(rows - row, 0, ROWS);
    left = cols > 0 && end > k ? (int)(end - k) : 0;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int b = q / Ld::kRounds;
      voff[q] = ld.offset(q % Ld::kRounds, (int)clamp64(cols - b * 128, 0, 128)) + b * 128 * (int)sizeof(T);
    }
  }
  __device__ inline void load(uint32_t dst) {
    const int n = left < K ? left : K;
    const int range = whole ? whole : ((n - 1) * (int)stride + cols) * (int)sizeof(T);
    load_lds16s<kLoads, NL * 16>(buffer_of(from, n > 0 ? range : 0), voff, dst);
    from += K * stride, left -= n;
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

template <typename T_, int WM_, int WN_, int TM_, int TN_, int KB_, bool TA, bool TB> struct Product {
  using T = T_;
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, KB = KB_;
  static constexpr int NL = 64 * WM * WN, BM = WM * TM * 32, BN = WN * TN * 32, K = KB / sizeof(T);
  using A = Side<T, BM, TA, NL, KB>;
  using B = Side<T, BN, TB, NL, KB>;
  static constexpr int kRing = 4, kStage = A::kBytes + B::kBytes, kLds = kRing * kStage;
  static constexpr int NT = KB / 32;  // steps of a stage
  static constexpr int kWaves = 2;      // that a SIMD has
  static_assert(kLds <= 160 * 1024, "");
  A a;
  B b;
  uint32_t lds0;
  int wave, lane, wm, wn;
  f32x16 acc[TM][TN];
  u32x4 x[2][TM], y[2][TN];

  __device__ inline void init(char* lds, int64_t sa, int64_t sb) {
    lds0 = uni((uint32_t)(size_t)(CUTBCE_LDS char*)lds);
    wave = uni(threadIdx.x / 64), lane = threadIdx.x % 64;
    wm = wave % WM, wn = wave / WM;
    a.init(sa), b.init(sb);
  }
  __device__ inline void clear() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};
  }
  __device__ inline uint32_t stage(int s) const { return lds0 + (uint32_t)(s & (kRing - 1)) * kStage; }
  // operand n of a step, in the order in which the products need them: TN of side b, then TM of side a
  __device__ inline void read(int q, int n, uint32_t at, int t) {
    if (n < TN) y[q][n] = B::op(at + A::kBytes, wn * TN + n, t, lane);
    else x[q][n - TN] = A::op(at, wm * TM + n - TN, t, lane);
  }
  __device__ inline void fetch(int s) {
    a.load(stage(s) + wave * 1024);
    b.load(stage(s) + A::kBytes + wave * 1024);
  }
  // The products of `turns` stages, which a and b have been started for; before(s) is called before stage s is loaded,
  // done(s) behind its products.
  template <typename F, typename D> __device__ inline void run(int turns, F before, D done) {
    constexpr int kLoads = A::kLoads + B::kLoads, OPS = TM + TN, MMAS = TM * TN;
    static_assert(OPS <= 2 * MMAS && (kRing - 2) * kLoads < 64, "");
    clear();
    wait_and_sync<>();  // (the ring's last readers are done, and what the waits below would count)
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) before(s), fetch(s);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((kRing - 2) * kLoads) : "memory");
#pragma unroll
    for (int n = 0; n < OPS; ++n) read(0, n, stage(0), 0);
    for (int s = 0; s < turns; ++s) {
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((kRing - 3) * kLoads) : "memory");
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t at = t + 1 < NT ? stage(s) : stage(s + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MMAS; ++m) {
          acc[m / TN][m % TN] = Mma<T>::mma(x[t & 1][m / TN], y[t & 1][m % TN], acc[m / TN][m % TN]);
#pragma unroll
          for (int n = m; n < OPS; n += MMAS) read((t + 1) & 1, n, at, (t + 1) % NT);
          if (t == 0 && m == 1) before(s + kRing - 1), fetch(s + kRing - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      done(s);
    }
    wait_and_sync<>();  // no load may reach LDS after the workgroup's end
  }
};

enum Tiling { kSmall, kLarge, kNarrow };
template <typename T, int TILING> struct Sizes {
  static constexpr int KB = 64;
  using Sums = Product<T, 2, 2, 2, 2, KB, false, false>;
  using Dh = Product<T, 2, 2, 2, 2, KB, false, true>;
  using De = Product<T, 2, 2, 2, 2, KB, true, true>;
};
template <> struct Sizes<__bf16, kLarge> {
  using Sums = Product<__bf16, 2, 4, 4, 2, 64, false, false>;
  using Dh = Product<__bf16, 2, 4, 4, 2, 64, false, true>;
  using De = Product<__bf16, 2, 4, 4, 2, 64, true, true>;
};
template <typename T> struct Sizes<T, kNarrow> : Sizes<T, kSmall> {
  using Sums = Product<T, 4, 1, 1, 2, 64, false, false>;
  using Dh = Product<T, 1, 4, 2, 1, 64, false, true>;
};
// Tiles of 256 x 256 are read by half as many workgroups, but leave CUs idle where there are few of them. 65,536
// items of 1,024 features, all four products: 200 rows 224 us in large tiles and 212 in small ones, 512 rows 366 and
// 410; 4,096 rows, 131,072 items of 2,048: 8.5 ms and 10.7. 4,149 rows, 392 items of 1,000, 34 large tiles: logits 37
// us, so 20. Up to 64 rows tiles are 64 rows wide, where half a small one would be empty (float32, 64 rows, 100,000 x
// 512: logits 143 us in small tiles and 83, dH 119 and 68; bf16 of 40,000 x 512: 15 and 13, 15 and 12). From 65 rows
// on two of them take what one small tile does (65 to 96 rows, all four products, small and narrow: float32 533 and
// 506 us, bf16 78 and 82).
inline Tiling tiling_of(int64_t R, int64_t V, int dtype) {
  if (R <= 64) return kNarrow;
  return dtype == 1 && R >= 512 && cdiv(R, 256) * cdiv(V, 256) >= 256 ? kLarge : kSmall;
}

// Tile (i, j) of ni x nj for a workgroup: every eighth workgroup, those of one XCD, has tiles next to each other, in
// blocks eight tiles wide, so that they read the same rows of both sides at about the same time. j is out of range for
// workgroups beyond the last tile.
struct TileAt {
  int i, j;
};
__device__ inline TileAt tile_at(int bid, int ni, int nj) {
  const int total = ni * nj, per = total / 8, more = total % 8, xcd = bid % 8;
  if (bid / 8 >= per + (xcd < more ? 1 : 0)) return {0, 0x7fffffff};  // (a grid for more rows than there are)
  const int u = xcd * per + (xcd < more ? xcd : more) + bid / 8;
  const int group = u / (8 * nj), wide = ni - group * 8 < 8 ? ni - group * 8 : 8, in = u - group * 8 * nj;
  return {group * 8 + in % wide, in / wide};
}

// How many of them a workgroup has that takes bid, bid + the grid, ... in turn (a grid that is a multiple of 8).
__device__ inline int tiles_at(int ni, int nj) {
  const int total = ni * nj, mine = total / 8 + ((int)blockIdx.x % 8 < total % 8 ? 1 : 0), first = blockIdx.x / 8;
  const int step = gridDim.x / 8;
  return mine > first ? (mine - first + step - 1) / step : 0;
}

// Units of work: tiles of rows x shares of the vocabulary, the shares' number from that of the tiles. Neighbouring
// units, which read the same items, go to workgroups of one XCD (every eighth).
struct Units {
  int tiles, shares;
};
__device__ inline Units units_of(int n, int64_t V, int bm, int bn, int grid) {
  Units u;
  u.tiles = (n + bn - 1) / bn;
  const int steps = (int)(((uint32_t)V + bm - 1) / bm);
  const int s = u.tiles ? grid / u.tiles : 1;
  u.shares = s < 1 ? 1 : (s > steps ? steps : s);
  return u;
}
template <typename P> constexpr int kCeGrid = P::kLds > 80 * 1024 ? 256 : 512;  // workgroups that are resident

// A unit's tiles follow one another without a pause in the loads. A lane has results of TN rows and keeps their running
// maximum (of z in base 2) and sum of exponentials; both halves of a wave join at the unit's end. The exponentials
// are not hidden: 128 a lane and tile, a third of the time at 512 features (4,096 rows x 262,144 x 512: 1,230 to
// 1,390 us, 0.79 to 0.89 PFLOP/s), a tenth at 2,048.
template <typename P>
__global__ __launch_bounds__(P::NL, P::kWaves) void k_ce_sums(Ce c, float2* __restrict__ part) {
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
  const int steps = (int)(((uint32_t)c.V + P::BM - 1) / P::BM);
  const int nk = (c.D + P::K - 1) / P::K, h = p.lane / 32;
  for (int k = blockIdx.x / 8; k < per; k += gridDim.x / 8) {
    const int u = (blockIdx.x % 8) * per + k;
    if (u >= total) break;
    const int tile = u % units.tiles, share = u / units.tiles;
    const Share part_of = share_at(steps, units.shares, share);
    const int64_t v0 = part_of.first, v1 = v0 + part_of.count;
    const int64_t row0 = (int64_t)tile * P::BN;
    float m[P::TN], s[P::TN];
    int target[P::TN];
#pragma unroll
    for (int j = 0; j < P::TN; ++j) {
      const int64_t i = row0 + (p.wn * P::TN + j) * 32 + p.lane % 32;
      m[j] = -INFINITY, s[j] = 0.f;
      target[j] = i < n ? targets[i] : -1;
    }
    int64_t fv = v0 * P::BM;  // the items whose stages are being loaded, and how many of those are left
    int fk = nk, left = nk;   // (left: of the tile that is being multiplied)
    int v = (int)(v0 * P::BM) + p.wm * P::TM * 32;
    p.a.start(E, fv, c.V, 0, c.D);
    p.b.start(H, row0, n, 0, c.D);
    p.run(
        (int)(v1 - v0) * nk,
        [&](int) {
          if (fk == 0) {
            fk = nk, fv += P::BM;
            p.a.start(E, fv, fv < v1 * P::BM ? c.V : 0, 0, c.D);
            p.b.start(H, row0, n, 0, c.D);
          }
          --fk;
        },
        [&](int) {
          if (--left) return;
          left = nk;
#pragma unroll
          for (int j = 0; j < P::TN; ++j) {
            if (__any((unsigned)(target[j] - v) < (unsigned)(P::TM * 32)) || (int64_t)v + P::TM * 32 > c.V) {
              // (compared with constants: a lane's items held as numbers would not fit the registers)
              const int hit = target[j] - v - 4 * h, end = (int)clamp64(c.V - v, 0, P::TM * 32) - 4 * h;
#pragma unroll
              for (int i = 0; i < P::TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const int item = i * 32 + acc_row(e, 0);
                  if (item == hit || item >= end) p.acc[i][j][e] = -INFINITY;
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
            float add[2] = {};
#pragma unroll
            for (int i = 0; i < P::TM; ++i)
#pragma unroll
              for (int e = 0; e < 16; ++e) add[e & 1] += exp2_of(__builtin_fmaf(p.acc[i][j][e], cc, -base));
            s[j] += add[0] + add[1];
          }
          p.clear();
          v += P::BM;
        });
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

// What a row's shares are, in the kernel that left their sums: k_ce_sums (slots for each share), or the sweep.
struct JoinHow {
  int bm, bn, grid, slots;
  __device__ inline int of(int n, int64_t V) const {
    if (!bm) return sweep_shares((n + bn - 1) / bn, sweep_stages(V), grid);
    return units_of(n, V, bm, bn, grid).shares * slots;
  }
};

// A wave has a row of the batch: joins its shares' sums.
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
  const int slots = how.of(at<CeHead>(c.saved, c.at.head)->n, c.V);
  const float2* mine = part + (int64_t)i * slots;
  const float z = zt[i];
  float m = z;
#pragma unroll 4
  for (int k = lane; k < slots; k += 64) m = top_of(m, mine[k]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  float others = 0.f;
#pragma unroll 4
  for (int k = lane; k < slots; k += 64) others += mine[k].y * share_of(mine[k], m);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) others += __shfl_xor(others, o, 64);
  if (lane == 0) finish_row(c, i, r, z, m, others, row_loss, each);
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

// dz of the piece in blocks of 64 bytes of items: [width / block][rows][block], rows = R rounded up to 32; zeros for
// items behind the vocabulary's end and for the rows from n to the next multiple of 32. A stage of the product with E
// is then one range of memory, and what a wave stores whole lines. In 16 bits the items of each 16 stand in the order
// 0-3, 8-11, 4-7, 12-15: a lane's eight results are next to each other, and are the operand of the product with E in
// the order in which the transposed reads of E give their items. (Rows of the piece's width instead, 64 KB apart: dH
// of 4,096 x 262,144 x 512 1,740 us, so 1,490.) A workgroup goes through its tiles without a pause in the loads (each
// tile a workgroup: dz 1,660 us, so 1,490). Storing the values in 16 bits rounds them by at most 2^-8 of themselves,
// as the product's operands are in any case; what that cuts off the targets' is added to both products
// (multiply_rests, k_ce_dh_join).
template <typename T> constexpr int kBlock = 64 / sizeof(T);
__host__ __device__ constexpr inline int item_at(int place) {  // of 16 bits
  return (place & ~12) | (place & 4) << 1 | (place & 8) >> 1;
}
template <typename P>
__global__ __launch_bounds__(P::NL, P::kWaves) void k_ce_dz(Ce c, int64_t v0, int64_t width,
                                                            typename P::T* __restrict__ dz) {
  using T = typename P::T;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int ni = (int)cdiv(n, P::BN), nj = (int)(width / P::BM), mine = tiles_at(ni, nj);
  P p;
  p.init(lds, c.D, c.D);
  const T *E = (const T*)c.E, *H = at<T>(c.saved, c.at.hc);
  const int nk = (c.D + P::K - 1) / P::K, h = p.lane / 32;
  const float cc = base2(c.scale);
  const int64_t rows = up(c.R, 32);
  int next = 0, fk = 0;          // the tile whose stages are loaded next, and how many of the one before are left
  int here = 0, left = nk;       // the tile that is being multiplied, and how many of its stages are left
  p.run(
      mine * nk,
      [&](int) {
        if (fk == 0) {
          const TileAt t = tile_at(blockIdx.x + next * gridDim.x, ni, nj);
          const bool any = next < mine;
          p.a.start(E, any ? v0 + (int64_t)t.j * P::BM : 0, any ? c.V : 0, 0, c.D);
          p.b.start(H, any ? (int64_t)t.i * P::BN : 0, any ? n : 0, 0, c.D);
          fk = nk, ++next;
        }
        --fk;
      },
      [&](int) {
        if (--left) return;
        left = nk;
        const TileAt t = tile_at(blockIdx.x + here * gridDim.x, ni, nj);
        ++here;
        const int64_t row0 = (int64_t)t.i * P::BN, v = v0 + (int64_t)t.j * P::BM;
#pragma unroll
        for (int j = 0; j < P::TN; ++j) {
          const int64_t i = row0 + (p.wn * P::TN + j) * 32 + p.lane % 32;
          if (i >= up(n, 32)) continue;
          float shift = INFINITY, own = 0.f;
          int64_t target = -1;
          if (i < n) {
            shift = at<float>(c.saved, c.at.shift)[i];
            own = at<float>(c.saved, c.at.own)[i];
            target = at<int32_t>(c.saved, c.at.target)[i];
          }
#pragma unroll
          for (int b = 0; b < P::TM; ++b) {
            const int64_t first = v + (p.wm * P::TM + b) * 32;
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = exp2_of(__builtin_fmaf(p.acc[b][j][e], cc, -shift));
            if (__any((uint64_t)(target - first) < 32u) || first + 32 > c.V) {
              const int hit = (int)clamp64(target - first, -1, 32) - 4 * h;
              const int end = (int)clamp64(c.V - first, 0, 32) - 4 * h;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int item = acc_row(e, 0);
                x[e] = item >= end ? 0.f : (item == hit ? own : x[e]);
              }
            }
            T* to = dz + ((first - v0) / kBlock<T> * rows + i) * kBlock<T>;
            if constexpr (sizeof(T) == 2) {
              store_vec(to + 8 * h, x);
              store_vec(to + 16 + 8 * h, x + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) store_vec(to + k / 2 * rows * kBlock<T> + k % 2 * 8 + 4 * h, x + 4 * k);
            }
          }
        }
        p.clear();
      });
}

// Parts of a long axis, of `steps` stages, for so many tiles: as many workgroups as are resident, each at least four
// stages.
__host__ __device__ inline int parts_of(int64_t tiles, int64_t steps, int grid) {
  int64_t parts = tiles < grid ? grid / (tiles ? (int)tiles : 1) : 1;
  if (parts > steps / 4) parts = steps / 4;
  return parts < 1 ? 1 : (int)parts;
}
// Of dH: by the rows that are counted, which only the device knows (777 rows, 739 of them counted, 65,537 x 256,
// float32: 275 us by all rows, 432 workgroups on 512 places; so 241). Of the numbers of parts that fill one turn of
// the resident workgroups, two, ... the first is taken that leaves at most 10% of them idle, or the best (296 tiles
// on 512 places, 4,697 rows, 202,265 x 1,000, float32: 25.8 ms in one part, 15.9 in five).
constexpr int kTurns = 4;
template <typename P> __host__ __device__ inline int64_t dh_tiles(int64_t n, int D) {
  return cdiv(n, P::BM) * cdiv(D, P::BN);
}
template <typename P> __host__ __device__ inline int64_t dh_most(int64_t width) {  // parts of at least four stages
  return width / P::K / 4 < 1 ? 1 : width / P::K / 4;
}
template <typename P> __host__ __device__ inline int dh_parts(int64_t n, int D, int64_t width) {
  const int grid = kCeGrid<P>;
  const int64_t all = dh_tiles<P>(n, D), most = dh_most<P>(width);
  if (all < 1 || all >= kTurns * grid) return 1;
  const int tiles = (int)all;
  int best = 1;
  float good = 0.f;
  for (int k = 1; k <= kTurns; ++k) {
    int p = k * grid / tiles;
    p = p < 1 ? 1 : (p > most ? (int)most : p);
    const float e = (float)(p * tiles) / (float)((p * tiles + grid - 1) / grid * grid);
    if (e > good) good = e, best = p;
    if (e >= 0.9f) break;
  }
  return best;
}

// sums[part][n][D] (+)= dz E over the part's items: rows x features, the first piece of the vocabulary writes.
template <typename P>
__global__ __launch_bounds__(P::NL, P::kWaves) void k_ce_dh(Ce c, int64_t v0, int64_t width, int first,
                                                    const typename P::T* __restrict__ dz, float* __restrict__ sums) {
  using T = typename P::T;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int cols = (c.D + P::BN - 1) / P::BN, rows = (int)cdiv(n, P::BM), parts = dh_parts<P>(n, c.D, width);
  const TileAt tile = tile_at(blockIdx.x, cols, rows * parts);  // (of one part of the items: neighbours read the same)
  if (!rows || tile.j >= rows * parts) return;
  const int part = tile.j / rows;
  const int64_t row0 = (int64_t)(tile.j % rows) * P::BM, d0 = (int64_t)tile.i * P::BN;
  P p;
  p.init(lds, 0, c.D);
  p.a.init_blocked(up(c.R, 32));
  const int64_t left = c.V - v0 < width ? c.V - v0 : width, steps = (left + P::K - 1) / P::K;
  const int64_t x0 = steps * part / parts, x1 = steps * (part + 1) / parts;
  const T* E = (const T*)c.E + v0 * c.D;
  p.a.start(dz, row0, n, x0 * P::K, x1 * P::K < width ? x1 * P::K : width);
  p.b.start(E, d0, c.D, x0 * P::K, x1 * P::K < left ? x1 * P::K : left);
  p.run((int)(x1 - x0), [](int) {}, [](int) {});
  float* to = sums + (int64_t)part * n * c.D;
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
__global__ __launch_bounds__(P::NL, P::kWaves) void k_ce_de(Ce c, int64_t v0, int64_t width, int parts,
                                                            const typename P::T* __restrict__ dz,
                                                            const float* __restrict__ grad,
                                                            typename P::T* __restrict__ dE, float* __restrict__ sums) {
  using T = typename P::T;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int cols = (c.D + P::BN - 1) / P::BN;
  const int64_t left = c.V - v0 < width ? c.V - v0 : width;
  const int items = (int)cdiv(left, P::BM);
  const TileAt tile = tile_at(blockIdx.x, cols, items * (PART ? parts : 1));
  if (tile.j >= items * (PART ? parts : 1)) return;
  const int part = PART ? tile.j / items : 0;
  const int64_t u0 = (int64_t)(PART ? tile.j % items : tile.j) * P::BM, d0 = (int64_t)tile.i * P::BN;
  P p;
  p.init(lds, 0, c.D);
  p.a.init_blocked(up(c.R, 32));
  const T* H = at<T>(c.saved, c.at.hc);
  const int64_t steps = (n + P::K - 1) / P::K;
  const int64_t x0 = PART ? steps * part / parts : 0, x1 = PART ? steps * (part + 1) / parts : steps;
  p.a.start_blocked(dz, u0 / kBlock<T>, up(c.R, 32), x0 * P::K, x1 * P::K < n ? x1 * P::K : n);
  p.b.start(H, d0, c.D, x0 * P::K, x1 * P::K < n ? x1 * P::K : n);
  p.run((int)(x1 - x0), [](int) {}, [](int) {});
  if constexpr (sizeof(T) == 2) {
    // what bf16 cut off the dz of this wave's items' own rows
    constexpr int kWide = P::TN * 32, kEach = kRests<kWide> + kRestList * 4;
    static_assert(P::WM * P::WN * kEach <= P::kLds && kEach % 256 == 0, "");
    const int64_t d = d0 + p.wn * kWide, last = x1 * P::K < n ? x1 * P::K : n;
    const uint32_t own = p.lds0 + p.wave * kEach, list = own + kRests<kWide>;
    for (int64_t next = d < c.D ? x0 * P::K : last; next < last;) {
      const int rests = list_rests(c, next, last, list, p.lane, [&](int t) {
        const int64_t place = t - (v0 + u0 + p.wm * P::TM * 32);
        return place >= 0 && place < P::TM * 32 ? (int)place : -1;
      });
      if (rests)
        multiply_rests<kWide, P::TM, 1>(
            c, H + d, (int)clamp64(c.D - d, 0, kWide), list, rests, item_at(p.lane % 32), own, p.lane,
            [&](int j, bf16x8 features, const u32x4* items) {
#pragma unroll
              for (int i = 0; i < P::TM; ++i)
                p.acc[i][j] = Mma<T>::mma(items[i], __builtin_bit_cast(u32x4, features), p.acc[i][j]);
            });
    }
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

// dH of all rows, zeros for those without a target: four features a lane, the sum of the parts', G lanes each.
template <typename P, int G>
__global__ __launch_bounds__(256) void k_ce_dh_join(Ce c, int64_t width, const float* __restrict__ sums,
                                                    const float* __restrict__ grad, typename P::T* __restrict__ dH) {
  using T = typename P::T;
  __shared__ f32x4 rest[G > 1 ? 256 : 1];
  constexpr int N = 256 / G;
  const int g = threadIdx.x / N;
  const int64_t x = ((int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * N + threadIdx.x % N) * 4;
  const bool there = x < c.R * c.D;
  const int64_t r = there ? x / c.D : 0;
  const int i = there ? at<int32_t>(c.saved, c.at.place)[r] : -1;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (i >= 0) {
    const int64_t from = (int64_t)i * c.D + (x - r * c.D);
    const int n = at<CeHead>(c.saved, c.at.head)->n, parts = dh_parts<P>(n, c.D, width);
#pragma unroll 4
    for (int k = g; k < parts; k += G) s += *(const f32x4*)(sums + (int64_t)k * n * c.D + from);
    if constexpr (sizeof(T) == 2) {
      if (g == 0) {  // what bf16 cut off the target's dz (multiply_rests has it for dE)
        const float own = at<float>(c.saved, c.at.own)[i], rest = own - (float)(__bf16)own;
        const int64_t target = at<int32_t>(c.saved, c.at.target)[i];
        const bf16x4 item = *(const bf16x4*)((const __bf16*)c.E + target * c.D + (x - r * c.D));
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += rest * (float)item[j];
      }
    }
  }
  if constexpr (G > 1) {
    rest[threadIdx.x] = s;
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int k = 1; k < G; ++k) s += rest[k * N + threadIdx.x];
  }
  if (!there) return;
  if (i >= 0) s *= *grad * c.scale;
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
  int de_parts;
  size_t dz, dh, de, bytes;  // offsets in the workspace
};
template <typename T, int TILING> Plan plan_of(int64_t R, int64_t V, int D) {
  using S = Sizes<T, TILING>;
  if (R < 1) R = 1;
  Plan p;
  // A piece's dz takes up to 512 MB, or that of 256 items. For each piece dH's partial sums are read and written
  // again, and the launches have their tails; what is beyond the 256 MB of the memory-side cache comes from memory.
  // Measured, dz + dH + dE of 4,096 x 262,144 x 512 in pieces of 64 MB, 256 MB, 1 GB: 5.6, 4.2, 3.8 ms; of 131,072 x
  // 2,048: 6.7, 6.2, 6.0.
  const int64_t rows = up(R, 32);
  int64_t width = ((int64_t)512 << 20) / (rows * (int64_t)sizeof(T)) / 256 * 256;
  if (width < 256) width = 256;
  if (width > up(V, 256)) width = up(V, 256);
  p.width = width;
  p.de_parts = parts_of(width / S::De::BM * cdiv(D, S::De::BN), cdiv(R, S::De::K), kCeGrid<typename S::De>);
  size_t b = 0;
  p.dz = b, b += up(rows * width * (int64_t)sizeof(T), 256);
  // dH's parts: one of all rows, or as many tiles as kTurns turns have
  int64_t few = (int64_t)kTurns * kCeGrid<typename S::Dh> * S::Dh::BM * (S::Dh::BN < D ? S::Dh::BN : D);
  if (few > dh_most<typename S::Dh>(width) * R * D) few = dh_most<typename S::Dh>(width) * R * D;
  p.dh = b, b += up((few > R * D ? few : R * D) * 4, 256);
  p.de = b, b += p.de_parts > 1 ? up((int64_t)p.de_parts * width * D * 4, 256) : 0;
  p.bytes = b;
  return p;
}

struct ForwardPlan {
  size_t zt, each, part, bytes;
};
template <typename T, int TILING> ForwardPlan forward_plan(int64_t R, int D, bool grad) {
  using P = typename Sizes<T, TILING>::Sums;
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
  f.part = b, b += up((tiles > kCeGrid<P> ? tiles : kCeGrid<P>) * P::BN * P::WM * 8, 256);
  f.bytes = b;
  return f;
}

template <typename T, int TILING>
hipError_t forward_t(const Ce& c, int id_bytes, const T* H, const void* targets, const float* weight, bool grad,
                     float* loss, float* row_loss, hipStream_t st) {
  using P = typename Sizes<T, TILING>::Sums;
  const ForwardPlan f = forward_plan<T, TILING>(c.R, c.D, grad);
  float *zt = (float*)(c.ws + f.zt), *each = (float*)(c.ws + f.each);
  float2* part = (float2*)(c.ws + f.part);
  const unsigned groups = (unsigned)(c.R < 16 ? 1 : c.R > 8192 ? 512 : cdiv(c.R, 16));
  if (id_bytes == 4) k_ce_rows<T, int32_t><<<groups, 1024, 0, st>>>(c, H, (const int32_t*)targets, weight, zt);
  else k_ce_rows<T, int64_t><<<groups, 1024, 0, st>>>(c, H, (const int64_t*)targets, weight, zt);
  const bool swept = ce_swept(c.D, c.dtype);
  if (swept && c.R) {
    const hipError_t e = launch_ce_rows(c, c.ws + f.part, grad, zt, row_loss, each, st);
    if (e != hipSuccess) return e;
  } else if (c.R) {
    const hipError_t e = allow_lds<k_ce_sums<P>>(P::kLds);
    if (e != hipSuccess) return e;
    k_ce_sums<P><<<kCeGrid<P>, P::NL, P::kLds, st>>>(c, part);
  }
  if (c.R && !(swept && grad)) {
    const JoinHow how =
        swept ? JoinHow{0, sweep_rows(c.D), sweep_grid(c.D), 1} : JoinHow{P::BM, P::BN, kCeGrid<P>, P::WM};
    k_ce_join<<<(unsigned)cdiv(c.R, 4), 256, 0, st>>>(c, how, part, zt, row_loss, each);
  }
  k_ce_loss<<<1, 1024, 0, st>>>(c, each, loss);
  return hipGetLastError();
}

template <typename T, int TILING>
hipError_t backward_t(const Ce& c, const float* grad, T* dH, T* dE, hipStream_t st) {
  using S = Sizes<T, TILING>;
  const Plan p = plan_of<T, TILING>(c.R, c.V, c.D);
  T* dz = (T*)(c.ws + p.dz);
  float *dh = (float*)(c.ws + p.dh), *de = (float*)(c.ws + p.de);
  hipError_t e = allow_lds<k_ce_dz<typename S::Sums>>(S::Sums::kLds);
  if (e == hipSuccess) e = allow_lds<k_ce_dh<typename S::Dh>>(S::Dh::kLds);
  if (e == hipSuccess) e = allow_lds<k_ce_de<typename S::De, false>>(S::De::kLds);
  if (e == hipSuccess) e = allow_lds<k_ce_de<typename S::De, true>>(S::De::kLds);
  if (e != hipSuccess) return e;
  for (int64_t v = 0; v < c.V; v += p.width) {
    const int64_t tiles = up(cdiv(c.R, S::Sums::BN) * (p.width / S::Sums::BM), 8);
    const unsigned grid = (unsigned)(tiles < kCeGrid<typename S::Sums> ? tiles : kCeGrid<typename S::Sums>);
    if (c.R) k_ce_dz<typename S::Sums><<<grid, S::Sums::NL, S::Sums::kLds, st>>>(c, v, p.width, dz);
    if (dH && c.R) {
      const int64_t one = dh_tiles<typename S::Dh>(c.R, c.D), turns = kTurns * kCeGrid<typename S::Dh>;
      int64_t most = one * dh_most<typename S::Dh>(p.width);  // workgroups, for any number of counted rows
      most = most > turns ? (one > turns ? one : turns) : most;
      k_ce_dh<typename S::Dh><<<(unsigned)up(most, 8), S::Dh::NL, S::Dh::kLds, st>>>(c, v, p.width, v == 0, dz, dh);
    }
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
  if (dH && c.R) {
    // many parts are joined by 16 lanes for each four features (32 rows, 100,000 x 128, float32, 512 parts: 126 us by
    // one lane, so 6)
    const bool many = dh_parts<typename S::Dh>(c.R, c.D, p.width) >= 16;
    const int64_t blocks = cdiv(c.R * c.D, many ? 64 : 1024), turns = cdiv(blocks, kMaxGrid);
    const dim3 grid((unsigned)cdiv(blocks, turns), (unsigned)turns);
    if (many) k_ce_dh_join<typename S::Dh, 16><<<grid, 256, 0, st>>>(c, p.width, dh, grad, dH);
    else k_ce_dh_join<typename S::Dh, 1><<<grid, 256, 0, st>>>(c, p.width, dh, grad, dH);
  }
  return hipGetLastError();
}

}  // namespace

CeSaved ce_saved(int64_t R, int64_t V, int D, int dtype) {
  CeSaved s;
  size_t b = 0;
  s.head = b, b += 256;
  size_t* each[] = {&s.rows, &s.place, &s.target, &s.shift, &s.own, &s.coef};
  for (size_t* x : each) *x = b, b += up(R * 4, 256);
  s.hc = b, b += up(R * D * (dtype ? 2 : 4), 256);
  s.dh = b, b += ce_swept(D, dtype) ? up(R * D * 4, 256) : 0;
  s.bytes = b;
  return s;
}

// f with the type and the tiling of a problem
template <typename F> auto by_sizes(int64_t R, int64_t V, int dtype, F f) {
  using std::integral_constant;
  const Tiling tiling = tiling_of(R, V, dtype);
  if (!dtype)
    return tiling == kNarrow ? f(0.f, integral_constant<int, kNarrow>{}) : f(0.f, integral_constant<int, kSmall>{});
  return tiling == kNarrow  ? f((__bf16)0.f, integral_constant<int, kNarrow>{})
         : tiling == kLarge ? f((__bf16)0.f, integral_constant<int, kLarge>{})
                            : f((__bf16)0.f, integral_constant<int, kSmall>{});
}

size_t ce_forward_bytes(int64_t R, int64_t V, int D, int dtype, bool want_grad) {
  const size_t own = by_sizes(R, V, dtype, [&](auto x, auto tiling) {
    return forward_plan<decltype(x), decltype(tiling)::value>(R, D, want_grad).bytes;
  });
  return own + (want_grad ? 0 : ce_saved(R, V, D, dtype).bytes);
}
size_t ce_backward_bytes(int64_t R, int64_t V, int D, int dtype) {
  if (ce_swept(D, dtype)) return ce_items_bytes(D);
  return by_sizes(R, V, dtype, [&](auto x, auto tiling) {
    return plan_of<decltype(x), decltype(tiling)::value>(R, V, D).bytes;
  });
}

hipError_t launch_ce_forward(const Ce& c, int id_bytes, const void* H, const void* targets, const float* weight,
                             bool want_grad, float* loss, float* row_loss, hipStream_t st) {
  return by_sizes(c.R, c.V, c.dtype, [&](auto x, auto tiling) {
    using T = decltype(x);
    return forward_t<T, decltype(tiling)::value>(c, id_bytes, (const T*)H, targets, weight, want_grad, loss, row_loss,
                                                 st);
  });
}
hipError_t launch_ce_backward(const Ce& c, const float* grad, void* dH, void* dE, hipStream_t st) {
  if (ce_swept(c.D, c.dtype)) return launch_ce_items(c, c.ws, grad, dH, dE, st);
  return by_sizes(c.R, c.V, c.dtype, [&](auto x, auto tiling) {
    using T = decltype(x);
    return backward_t<T, decltype(tiling)::value>(c, grad, (T*)dH, (T*)dE, st);
  });
}

}  // namespace cutbce
