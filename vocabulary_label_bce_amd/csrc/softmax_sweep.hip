// Softmax cross entropy in two sweeps, for bfloat16 rows of up to 256 features: neither the logits nor their gradients
// leave the registers.
//
// Forward: a wave owns 64 rows (as two blocks of 32; beyond 128 features one block) and sweeps a share of the
// vocabulary, 32 items a step:
//   Z^T = E_step H^T,  P = exp2(c Z - ref),  sums += P,  dH^T += E_step^T P     (ref a row's reference)
// Backward: a wave owns as many items and sweeps all rows:
//   Z = H_step E^T,  P = w/W exp2(c Z - lse),  dE^T += H_step^T P
// A step's results have the owned rows (or items) as columns, so that a lane has values of one of them, and P is the
// second product's operand as it stands; the step's own tile, read row by row and transposed, is the other operand of
// both.
//
// Two blocks a wave halve what is read from LDS for a product: with one, LDS delivers 128 bytes a cycle at the matrix
// units' full rate, all that it can. Beyond 64 features they take all of a SIMD's registers for one wave, so the
// products have to hide the vector instructions of the same wave: in one turn of the loop the products Z of the next
// step and the gradient's of the step before run while the exponentials of this step are formed, none depending on
// another. The order is pinned, a share of the vector work behind each matrix instruction. Up to 64 features two
// workgroups fit a CU, and their waves hide each other (kPlain): a step's products, exponentials and products follow
// one another, which needs fewer registers (the backward's sweep of 5,120 rows and 100,000 items of 64 in turns as
// above, one wave a SIMD: 236 us, so 157, which with the rests of the targets are 160 to 180; the forward's 168
// either way).
//
// What bounds them: the matrix units' power. 14,336 rows x 876,000 x 128: 5.0 to 5.8 ms a sweep, 1.1 to 1.28 PFLOP/s at
// 1.5 to 1.8 GHz, a large product of the library having 1.30 on the same card. At 64 features an exponential costs as
// much as its products (770 to 840 TFLOP/s), at 256 a wave has one block (4,096 rows x 131,072: 1.05 ms for both,
// 1.05 PFLOP/s).
#include "softmax.h"

namespace cutbce {

namespace {

#define INLINED __attribute__((always_inline))

// Blocks of 32 that a wave owns; the ring's stages in LDS; and how many stages early a stage's loads are issued.
template <int DP> constexpr int kBlocks = DP > 128 ? 1 : 2;
template <int DP> constexpr int kStages = DP > 128 ? 4 : 5;
template <int DP> constexpr int kAhead = kStages<DP> - 2;
__host__ __device__ constexpr inline int items_grid(int D) { return D <= 64 ? 512 : 256; }  // of the backward
constexpr float kMost = 0x1p80f;              // sums of exponentials beyond which a row takes a new reference

__device__ inline uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Waves a SIMD has: two where the registers allow it.
template <int DP, bool ITEMS> constexpr int kWaves = DP <= 64 ? 2 : 1;

// The ring of one workgroup and a wave's operands.
template <int DP, bool AUX, bool GRAD> struct Sweep {
  using Ti = Tile<__bf16, DP>;
  using Ld = Dma<__bf16, DP, kSweepStage, 256>;
  using M = Mma<__bf16>;
  static constexpr int NT = Ti::kNT, NDB = Ti::kNDB;            // steps of Z's product; blocks of features
  static constexpr int kNB = kBlocks<DP>, kOwned = 4 * kNB * 32;  // a wave's blocks; what a workgroup owns
  static constexpr int kStages = cutbce::kStages<DP>, kAhead = cutbce::kAhead<DP>;
  static constexpr int kRow = Ti::kRowB, kTile = Ld::kBytes;    // bytes
  static constexpr int kAux = AUX ? 1024 : 0;                   // three arrays of 64 values, and room for a fourth
  static constexpr int kStage = kTile + kAux, kLds = kStages * kStage;
  static constexpr int kLoads = Ld::kRounds + (AUX ? 1 : 0);    // of a wave for a stage
  static constexpr bool kAlone = kWaves<DP, AUX> == 1 && GRAD, kHeld = kWaves<DP, AUX> == 1;
  static constexpr bool kPlain = !kHeld;  // one product after the other
  static_assert(NT == 2 * NDB, "");

  Ld ld;
  uint32_t lds0;
  int wave, lane, h;
  const __bf16* X;       // the streamed rows
  int64_t rows, from;    // how many there are; the first of this share
  int D;
  u32x4 own[kNB][NT];    // the owned rows
  u32x4 x[NT];           // a step's rows
  bf16x8 t[NT];          // a step's rows, transposed
  f32x16 z[2][kNB];      // of the steps in turn
  uint32_t p[2][kNB][8];
  f32x16 acc[NDB][kNB];
  uint32_t row_off, col_off;
  uint32_t ra[NT], ca[NT];

  __device__ inline void init(char* lds, const __bf16* X_, int64_t rows_, int D_) {
    lds0 = uni((uint32_t)(size_t)(CUTBCE_LDS char*)lds);
    wave = uni(threadIdx.x / 64), lane = threadIdx.x % 64, h = lane / 32;
    X = X_, rows = rows_, D = D_;
    ld.init(threadIdx.x, D);
    row_off = base_row<__bf16, DP>(0, lane), col_off = M::template base_t<DP>(0, lane);
  }
  __device__ inline uint32_t slot(int s) const { return lds0 + (uint32_t)(s % kStages) * kStage; }
  __device__ static inline uint32_t step_of(int s) {  // from stage s's place in the ring to that of the next
    return s % kStages == kStages - 1 ? (uint32_t)-((kStages - 1) * kStage) : (uint32_t)kStage;
  }
  // The wave's loads of a stage from `range` to LDS byte `dst`, as load_lds16 does them one by one.
  __device__ inline void load_stage(u32x4 range, uint32_t dst) const {
    static_assert(Ld::kRounds == 2 || Ld::kRounds == 4 || Ld::kRounds == 8, "");
    if constexpr (Ld::kRounds == 8) {
      load_four(range, dst, 0);
      load_four(range, dst + 0x4000, 4);
    } else if constexpr (Ld::kRounds == 4) {
      load_four(range, dst, 0);
    } else {
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
                   "s_add_u32 m0, m0, 0x1000\n\ts_nop 1\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
                   :: "s"(uni(dst)), "v"(ld.offset(0, D)), "v"(ld.offset(1, D)), "s"(range) : "m0", "scc");
    }
  }
  __device__ inline void load_four(u32x4 range, uint32_t dst, int q) const {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, 0x1000\n\ts_nop 1\n\tbuffer_load_dwordx4 %2, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, 0x1000\n\ts_nop 1\n\tbuffer_load_dwordx4 %3, %5, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, 0x1000\n\ts_nop 1\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                 :: "s"(uni(dst)), "v"(ld.offset(q, D)), "v"(ld.offset(q + 1, D)), "v"(ld.offset(q + 2, D)),
                    "v"(ld.offset(q + 3, D)), "s"(range) : "m0", "scc");
  }
  template <int STEP> __device__ inline void load_owned(const __bf16* base, int64_t first, int64_t n) {
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
      const int64_t i = first + (b * 32 + lane % 32) * STEP;
      load_own<__bf16, DP>(own[b], base + i * D, i < n, D, lane);
    }
  }
  __device__ inline void clear() {
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
#pragma unroll
      for (int d = 0; d < NDB; ++d) acc[d][b] = f32x16{};
#pragma unroll
      for (int i = 0; i < 8; ++i) p[1][b][i] = 0;
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) t[k] = bf16x8{};
  }
  // Z's product of a step (x is then free): into z[to]
  __device__ inline void first(int to) {
#pragma unroll
    for (int b = 0; b < kNB; ++b) z[to][b] = f32x16{};
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int b = 0; b < kNB; ++b) z[to][b] = M::mma(x[k], own[b][k], z[to][b]);
  }
  __device__ inline void read_rows(uint32_t at) {
#pragma unroll
    for (int k = 0; k < NT; ++k) x[k] = load_row(at + row_off, k);
  }
  __device__ inline bf16x8 operand(int q, int b, int g) const {
    const uint32_t* x = p[q][b] + 4 * g;
    return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], x[2], x[3]});
  }
  __device__ inline void gradient(int q, int k, int b) {  // the k-th of NT parts of the product with p[q]
    if constexpr (GRAD)
      acc[k % NDB][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(t[k], operand(q, b, k / NDB), acc[k % NDB][b], 0, 0, 0);
  }
  // Where a SIMD has one wave, the products' sums stay in accumulation registers (left alone, the compiler moves all of
  // them to the others and back in every turn, for the rare branch that rescales them), and results are read from there
  // one by one, each in its place.
  __device__ inline void settle() {
    if constexpr (GRAD && kAlone) {
#pragma unroll
      for (int d = 0; d < NDB; ++d)
#pragma unroll
        for (int b = 0; b < kNB; ++b) asm volatile("" : "+a"(acc[d][b]));
    }
  }
  __device__ inline float result(int q, int b, int e) {
    if constexpr (kAlone) asm volatile("" : "+a"(z[q][b]));
    return z[q][b][e];
  }
  // LDS addresses of the reads ahead: of the rows from stage `next` on, of the transposed rows from stage `here` on.
  // They are moved on from stage to stage, an addition each.
  __device__ inline void aim(uint32_t next, uint32_t here) {
    if constexpr (!kHeld) {
      ra[0] = next + row_off, ca[0] = here + col_off;
      return;
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      ra[k] = (next + row_off) ^ (2 * k * 16);
      const int db = k % NDB, e = k / NDB;
      ca[k] = (here + col_off) ^ (((db * 4) ^ Ti::swz(8 * e)) * 16);
    }
  }
  __device__ inline void move_on(uint32_t by_next, uint32_t by_here) {
#pragma unroll
    for (int k = 0; k < (kHeld ? NT : 1); ++k) ra[k] += by_next, ca[k] += by_here;
  }
  __device__ inline uint32_t row_at(int k) const { return kHeld ? ra[k] : ra[0] ^ (2 * k * 16); }
  __device__ inline uint32_t col_at(int db, int e) const {
    return kHeld ? ca[e * NDB + db] : ca[0] ^ (((db * 4) ^ Ti::swz(8 * e)) * 16);
  }
  template <int Q> __device__ inline void read_row(int k) { x[k] = lds16(row_at(k) + Q * 32 * kRow); }
  template <int Q> __device__ inline void read_col(int k) {
    const int db = k % NDB, g = k / NDB;
    s16x4 y[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      y[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (CUTBCE_LDS s16x4*)(size_t)(col_at(db, e) + (Q * 32 + 16 * g + 8 * e) * kRow));
    t[k] = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(y[0], y[1], 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // One turn: Z of the next step, the gradient's product of the step before, and work(0 .. kSlots - 1) in between, a
  // share of the vector instructions behind each matrix instruction: they run beside it, and the next one waits for
  // them. Reads ahead: the rows of the step after the next, the transposed rows of this step.
  static constexpr int kSlots = (GRAD ? 2 : 1) * NT * kNB;
  template <int Q, typename F> __device__ inline void turn(F work) {
    settle();
#pragma unroll
    for (int b = 0; b < kNB; ++b) z[1 - Q][b] = f32x16{};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        z[1 - Q][b] = M::mma(x[k], own[b][k], z[1 - Q][b]);
        if (b == kNB - 1) read_row<Q>(k);
        work((k * kNB + b) * (GRAD ? 2 : 1));
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (GRAD) {
          gradient(1 - Q, k, b);
          if (b == kNB - 1) read_col<Q>(k);
          work((k * kNB + b) * 2 + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  // The exponentials of step Q's results, element e = i / kNB of block b = i % kNB in turn: one is begun in its slot,
  // and added and packed in later ones, when it is there. argument(b, e, z) gives the exponent.
  template <int Q, typename A> __device__ inline void element(int i, float* y, A argument) {
    y[i & 3] = exp2_of(argument(i % kNB, i / kNB, result(Q, i % kNB, i / kNB)));
  }
  template <int Q> __device__ inline void finished(int i, const float* y) {
    const int b = i % kNB, e = i / kNB;
    if (e & 1) {
      p[Q][b][e / 2] = pack2(y[(i - kNB) & 3], y[i & 3]);
      // (here: the compiler would move what is not needed before the next turn)
      asm volatile("" : "+v"(p[Q][b][e / 2]));
    }
  }
  // The last step's part of the gradient.
  __device__ inline void last(int q) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int b = 0; b < kNB; ++b) gradient(q, k, b);
  }
};

template <int N> __device__ inline void landed_and_sync() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------------------------------------------------
// Forward. part[row * shares + share]: the row's reference and the sum of its exponentials, its target left out;
// sums[share][row]: those of the products.
// ---------------------------------------------------------------------------------------------------------
//
// A row's reference is the largest of its first step. It holds unless logits rise by 55 above that, or none of those
// items counts, or something is not finite: the unit is then marked in `off`, and a second launch (CAREFUL) goes
// through the marked ones again, one product after the other, a row whose exponentials have grown taking its largest
// as reference. The unit's other rows go through the same numbers again: what a row gets does not depend on the
// others.
template <int DP, bool GRAD, bool CAREFUL>
__global__ __launch_bounds__(256, (kWaves<DP, false>)) void k_ce_sweep_rows(Ce c, float2* __restrict__ part,
                                                                   float* __restrict__ sums, int* __restrict__ off) {
  using S = Sweep<DP, false, GRAD>;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int tiles = (n + S::kOwned - 1) / S::kOwned;
  const int stages = sweep_stages(c.V);
  const int shares = sweep_shares(tiles, stages, sweep_grid(c.D)), total = tiles * shares, per = (total + 7) / 8;
  const float cc = base2(c.scale);
  const int32_t* targets = at<int32_t>(c.saved, c.at.target);
  S s;
  s.init(lds, (const __bf16*)c.E, c.V, c.D);
  for (int unit = blockIdx.x / 8; unit < per; unit += gridDim.x / 8) {
    const int u = (blockIdx.x % 8) * per + unit;  // neighbours, on one XCD, read the same items
    if (u >= total) break;
    if (CAREFUL && !off[u]) continue;
    const int tile = u % tiles, share = u / tiles;
    const Share part_of = share_at(stages, shares, share);
    const int64_t s0 = part_of.first;
    const int count = part_of.count;
    const int64_t own0 = (int64_t)tile * S::kOwned + s.wave * (S::kNB * 32);
    wait_and_sync<>();  // (the ring's last readers are done, and stores, which the waits below would count)
    s.template load_owned<1>(at<__bf16>(c.saved, c.at.hc), own0, n);
    int target[S::kNB];
    float ref[S::kNB], sum[S::kNB];
#pragma unroll
    for (int b = 0; b < S::kNB; ++b) {
      const int64_t i = own0 + b * 32 + s.lane % 32;
      target[b] = i < n ? targets[i] : -1;
    }
    auto fetch = [&](int k) INLINED {
      const int64_t row = (s0 + k) * kSweepStage;
      const u32x4 r = s.ld.range(s.X + row * c.D, k < count ? c.V - row : 0, c.D, c.D);
      s.load_stage(r, s.slot(k) + s.wave * 1024);
    };
    auto start = [&]() INLINED {
      s.clear();
#pragma unroll
      for (int k = 0; k < S::kAhead; ++k) fetch(k);
      landed_and_sync<(S::kAhead - 1) * S::kLoads>();
      s.read_rows(s.slot(0));
      s.first(0);
    };
    // leaves out of step Q of stage k what is a row's target or past the vocabulary's end
    auto leave_out = [&](auto half, int k) INLINED {
      constexpr int Q = decltype(half)::value;
      const int item0 = (int)((s0 + k) * kSweepStage) + Q * 32;
      bool rare = item0 + 32 > c.V;
#pragma unroll
      for (int b = 0; b < S::kNB; ++b) rare |= (unsigned)(target[b] - item0) < 32u;
      if (__builtin_expect(__any(rare), 0)) {
#pragma unroll
        for (int b = 0; b < S::kNB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int item = item0 + acc_row(e, s.h);
            if (item == target[b] || item >= c.V) s.z[Q][b][e] = -INFINITY;
          }
      }
    };
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, 1>;
    // the first step's largest
    auto begin = [&]() INLINED {
      leave_out(Even{}, 0);
#pragma unroll
      for (int b = 0; b < S::kNB; ++b) {
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s.z[0][b][e]);
        top = fmaxf(top, other_half(top)) * cc;
        ref[b] = top > -INFINITY ? top : 0.f;
        sum[b] = 0.f;
      }
    };
    start();
    begin();
    if constexpr (!CAREFUL) {
      s.read_rows(s.slot(0) + (S::kPlain ? 0 : 32 * S::kRow));
      s.aim(s.slot(1), s.slot(0));
      auto step = [&](auto half, int k) INLINED {
        constexpr int Q = decltype(half)::value;
        float add[S::kNB][2] = {};
        if constexpr (S::kPlain) {
          s.first(Q);
          if (Q == 0) fetch(k + S::kAhead);
          s.read_rows(Q == 0 ? s.slot(k) + 32 * S::kRow : s.slot(k + 1));
          if constexpr (GRAD) {
#pragma unroll
            for (int n = 0; n < S::NT; ++n) s.template read_col<Q>(n);
          }
        }
        leave_out(half, k);
        float y[4];
        constexpr int ALL = S::kNB * 16;
        if constexpr (S::kPlain) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int b = 0; b < S::kNB; ++b) {
              float v[2];
#pragma unroll
              for (int j = 0; j < 2; ++j)
                add[b][j] += v[j] = exp2_of(__builtin_fmaf(s.z[Q][b][2 * i + j], cc, -ref[b]));
              if constexpr (GRAD) s.p[Q][b][i] = pack2(v[0], v[1]);
            }
          if constexpr (GRAD) s.last(Q);
        } else {
          auto end = [&](int i) {
            float& a = add[i % S::kNB][i / S::kNB & 1];
            a += y[i & 3];
            asm volatile("" : "+v"(a));
            if (GRAD) s.template finished<Q>(i, y);
          };
          s.template turn<Q>([&](int w) {
            if (Q == 0 && w == 1) fetch(k + S::kAhead);
#pragma unroll
            for (int i = ALL * w / S::kSlots; i < ALL * (w + 1) / S::kSlots; ++i) {
              s.template element<Q>(i, y, [&](int b, int, float z) { return __builtin_fmaf(z, cc, -ref[b]); });
              if (i) end(i - 1);
            }
          });
          end(ALL - 1);
        }
#pragma unroll
        for (int b = 0; b < S::kNB; ++b) sum[b] += add[b][0] + add[b][1];
      };
      s.settle();
      for (int k = 0; k < count; ++k) {
        landed_and_sync<(S::kAhead - 2) * S::kLoads>();  // stage k + 1 is there
        step(Even{}, k);
        step(Odd{}, k);
        s.move_on(S::step_of(k + 1), S::step_of(k));
        s.settle();
      }
      if constexpr (!S::kPlain) s.last(1);
      bool bad = false;
#pragma unroll
      for (int b = 0; b < S::kNB; ++b) bad |= !(sum[b] <= kMost) || !(sum[b] + other_half(sum[b]) >= 0.5f);
      bad = __syncthreads_or(bad);
      if (threadIdx.x == 0) off[u] = bad;
    } else {
      auto careful = [&](auto half, int k) INLINED {
        constexpr int Q = decltype(half)::value;
        if (Q == 1 || k > 0) {
          s.read_rows(s.slot(k) + Q * 32 * S::kRow);
          s.first(Q);
          leave_out(half, k);
        }
#pragma unroll
        for (int b = 0; b < S::kNB; ++b) {
          for (int again = 0; again < 2; ++again) {
            float add[2] = {};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float y[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) add[j] += y[j] = exp2_of(__builtin_fmaf(s.z[Q][b][2 * i + j], cc, -ref[b]));
              s.p[Q][b][i] = pack2(y[0], y[1]);
            }
            const uint64_t over = __ballot(!(add[0] + add[1] <= kMost) || !(sum[b] <= kMost));
            if (again || !over) {
              sum[b] += add[0] + add[1];
              break;
            }
            if (!((over >> s.lane | over >> (s.lane ^ 32)) & 1)) continue;
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s.z[Q][b][e]);
            top = fmaxf(top, other_half(top)) * cc;
            const float next = fmaxf(ref[b], top), f = exp2_of(ref[b] - next);
            ref[b] = next;
            sum[b] *= f;
            if constexpr (GRAD) {
#pragma unroll
              for (int d = 0; d < S::NDB; ++d) s.acc[d][b] *= f;
            }
          }
        }
        if constexpr (GRAD) {
          s.aim(s.slot(k), s.slot(k));
#pragma unroll
          for (int n = 0; n < S::NT; ++n) s.template read_col<Q>(n);
          s.last(Q);
        }
      };
      for (int k = 0; k < count; ++k) {
        if (k) landed_and_sync<(S::kAhead - 1) * S::kLoads>();
        careful(Even{}, k);
        careful(Odd{}, k);
        wait_and_sync<(S::kAhead - 1) * S::kLoads>();  // (the stage's place is read out)
        fetch(k + S::kAhead);
      }
    }
    wait_and_sync<>();  // no load may reach LDS after the unit's end
#pragma unroll
    for (int b = 0; b < S::kNB; ++b) {
      const int64_t i = own0 + b * 32 + s.lane % 32;
      const float whole = sum[b] + other_half(sum[b]);
      if (i >= n) continue;
      if (s.lane < 32) part[i * shares + share] = make_float2(ref[b], whole);
      if constexpr (GRAD) {
        f32x16 o[S::NDB];
#pragma unroll
        for (int d = 0; d < S::NDB; ++d) o[d] = s.acc[d][b];
        store_row<float, S::NDB>(sums + ((int64_t)share * n + i) * c.D, o, 1.f, c.D, s.lane);
      }
    }
  }
}

// A row of the batch: joins its shares' sums, and products into saved's dH (without the cotangent and scale). Without
// products k_ce_join does it. A workgroup has a row where rows are few and have many shares, else a wave has one.
template <bool WAVE>
__global__ __launch_bounds__(256) void k_ce_sweep_join(Ce c, const float2* __restrict__ part,
                                                       const float* __restrict__ sums, const float* __restrict__ zt,
                                                       float* __restrict__ row_loss, float* __restrict__ each) {
  __shared__ float4 rest[WAVE ? 1 : 256];
  constexpr int LANES = WAVE ? 64 : 256;
  const int tid = threadIdx.x % LANES, lane = tid % 64;
  const int64_t r = WAVE ? (int64_t)blockIdx.x * 4 + threadIdx.x / 64 : blockIdx.x;
  if (r >= c.R) return;
  const int i = at<int32_t>(c.saved, c.at.place)[r];
  if (i < 0) {
    if (tid == 0 && row_loss) row_loss[r] = 0.f;
    return;
  }
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const int shares = sweep_shares((n + sweep_rows(c.D) - 1) / sweep_rows(c.D), sweep_stages(c.V), sweep_grid(c.D));
  const float z = zt[i];
  const float2* mine_part = part + (int64_t)i * shares;
  float m = z;
  for (int k = lane; k < shares; k += 64) m = top_of(m, mine_part[k]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  float others = 0.f;
  for (int k = lane; k < shares; k += 64) others += mine_part[k].y * share_of(mine_part[k], m);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) others += __shfl_xor(others, o, 64);
  const float sum = others + exp2_of(z - m);
  if (tid == 0) finish_row(c, i, r, z, m, others, row_loss, each);
  // a group of DL lanes has the row's features, four each; the groups share the shares
  const int DL = c.D / 4, groups = LANES / DL, g = tid / DL, d = tid % DL * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (g < groups) {
#pragma unroll 4
    for (int k = g; k < shares; k += groups)
      s += *(const f32x4*)(sums + ((int64_t)k * n + i) * c.D + d) * share_of(mine_part[k], m);
  }
  if constexpr (WAVE) {
    const f32x4 own = s;
    for (int k = 1; k < groups; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += __shfl(own[j], (k * DL + lane) & 63, 64);
  } else {
    rest[tid] = make_float4(s[0], s[1], s[2], s[3]);
    __syncthreads();
    for (int k = 1; k < groups && g == 0; ++k) {
      const float4 x = rest[k * DL + tid];
      s += f32x4{x.x, x.y, x.z, x.w};
    }
  }
  if (g == 0) {
    const float coef = at<float>(c.saved, c.at.coef)[i];
    const __bf16* item = (const __bf16*)c.E + (int64_t)at<int32_t>(c.saved, c.at.target)[i] * c.D + d;
    float* to = at<float>(c.saved, c.at.dh) + (int64_t)i * c.D + d;
#pragma unroll
    for (int j = 0; j < 4; ++j) to[j] = coef * ((s[j] - others * (float)item[j]) / sum);
  }
}

// ---------------------------------------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------------------------------------

// The work, tiles of items (in steps of `spread`) x stages of rows, is one line that is cut into as many equal parts
// as there are workgroups (each at least kLeast stages, where there is that much): a workgroup goes through whole
// tiles, and the ends of its part are pieces of tiles that it shares with its neighbours. A piece's sums go to place
// 0 of its workgroup's two if it begins where the part does, else to 1, and are joined by k_ce_finish. (With whole
// tiles alone 391 tiles of 100,000 items on 256 CUs would take the time of 512.)
constexpr int kLeast = 4, kListBytes = 16 + kRestList * 4;
struct Line {
  int64_t stages, total;  // of a tile, and of all
  int parts;
  __device__ inline Line(int n, int64_t V, int D) {
    stages = n > 0 ? cdiv(n, kSweepStage) : 1;
    total = cdiv(V, sweep_rows(D)) * stages;
    const int grid = items_grid(D);
    parts = (int)(total / kLeast < grid ? (total < kLeast ? 1 : total / kLeast) : grid);
  }
  __device__ inline int64_t begin(int part) const { return total * part / parts; }
};

template <int DP>
__global__ __launch_bounds__(256, (kWaves<DP, true>)) void k_ce_sweep_items(Ce c, const float* __restrict__ grad,
                                                                            int64_t spread, __bf16* __restrict__ dE,
                                                                            float* __restrict__ sums) {
  using S = Sweep<DP, true, true>;
  extern __shared__ __align__(1024) char lds[];
  const int n = at<CeHead>(c.saved, c.at.head)->n;
  const float cc = base2(c.scale);
  const Line line(n, c.V, c.D);
  if ((int)blockIdx.x >= line.parts) return;
  const int64_t from = line.begin(blockIdx.x), to = line.begin(blockIdx.x + 1), tiles = cdiv(c.V, S::kOwned);
  S s;
  s.init(lds, at<__bf16>(c.saved, c.at.hc), n, c.D);
  const int32_t* targets = at<int32_t>(c.saved, c.at.target);
  const void* aux = s.wave == 1 ? (const void*)targets : c.saved + (s.wave == 2 ? c.at.own : c.at.shift);
  for (int64_t x = from; x < to;) {
    const int64_t at_tile = x / line.stages, tile = at_tile * spread % tiles;
    const int s0 = (int)(x - at_tile * line.stages);
    const int count = (int)(line.stages - s0 < to - x ? line.stages - s0 : to - x);
    const bool whole = count == line.stages;
    const int place = x == from ? 0 : 1;
    x += count;
    // The tile's items are dealt to the four waves one by one: neighbours, often targets together, go to different ones
    // (5,120 rows, 100,000 x 64, targets by popularity: 64 neighbours a wave 200 us, so 178).
    const int64_t own0 = tile * S::kOwned + s.wave;
    constexpr int kPlaces = (S::kOwned / 4 - 1) * 4;  // bits of an item that say which one of a wave's it is
    wait_and_sync<>();  // (the ring's last readers are done, and stores, which the waits below would count)
    s.template load_owned<4>((const __bf16*)c.E, own0, c.V);
    s.clear();
    auto fetch = [&](int k) INLINED {
      const int64_t row = (int64_t)(s0 + k) * kSweepStage;
      const int64_t left = k < count ? n - row : 0;
      const u32x4 r = s.ld.range(s.X + row * c.D, left, c.D, c.D);
      s.load_stage(r, s.slot(k) + s.wave * 1024);
      load_lds4(buffer_of((const char*)aux + row * 4, (int)clamp64(left, 0, kSweepStage) * 4), s.lane * 4,
                s.slot(k) + S::kTile + s.wave * 256);
    };
#pragma unroll
    for (int k = 0; k < S::kAhead; ++k) fetch(k);
    landed_and_sync<(S::kAhead - 1) * S::kLoads>();
    s.read_rows(s.slot(0));
    if constexpr (!S::kPlain) {
      s.first(0);
      s.read_rows(s.slot(0) + 32 * S::kRow);
    }
    // The wave's list of rows whose target it has: the row from which on it was full, the entries; and their number,
    // with 2 kRestList added when it is full.
    const uint32_t list = s.lds0 + S::kLds + s.wave * kListBytes;
    int listed = 0;
    f32x4 sh[4];
    // the shifts of a step (four at a time, as the ones before are done with) and, a row a lane, its targets
    auto shifts_at = [&](uint32_t at) INLINED {
      at += 16 * s.h;
      asm volatile("" : "+v"(at));
      return at;
    };
    auto read_shift = [&](int k, uint32_t at) INLINED { sh[k] = *(CUTBCE_LDS const f32x4*)(size_t)(at + 32 * k); };
    auto read_target = [&](uint32_t at) { return *(CUTBCE_LDS const int*)(size_t)(at + 256 + (s.lane % 32) * 4); };
#pragma unroll
    for (int k = 0; k < 4; ++k) read_shift(k, shifts_at(s.slot(0) + S::kTile));
    int t_next = read_target(s.slot(0) + S::kTile);
    s.aim(s.slot(1), s.slot(0));
    auto step = [&](auto half, int k) INLINED {
      constexpr int Q = decltype(half)::value;
      const uint32_t ax = s.slot(k) + S::kTile + Q * 128, after = Q == 0 ? ax + 128 : s.slot(k + 1) + S::kTile;
      const uint32_t shifts = shifts_at(after);
      const int t = t_next;
      float y[4];
      constexpr int ALL = S::kNB * 16;
      if constexpr (S::kPlain) {
        s.first(Q);
        if (Q == 0) fetch(k + S::kAhead);
        s.read_rows(Q == 0 ? s.slot(k) + 32 * S::kRow : s.slot(k + 1));
        t_next = read_target(after);
#pragma unroll
        for (int n = 0; n < S::NT; ++n) s.template read_col<Q>(n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
          for (int b = 0; b < S::kNB; ++b) {
            float v[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
              v[j] = exp2_of(__builtin_fmaf(s.z[Q][b][2 * i + j], cc, -sh[i / 2][2 * i % 4 + j]));
            s.p[Q][b][i] = pack2(v[0], v[1]);
          }
          if (i % 2) read_shift(i / 2, shifts);
        }
      } else {
        s.template turn<Q>([&](int w) {
          if (Q == 0 && w == 1) fetch(k + S::kAhead);
          if (w == 2) t_next = read_target(after);
#pragma unroll
          for (int i = ALL * w / S::kSlots; i < ALL * (w + 1) / S::kSlots; ++i) {
            s.template element<Q>(i, y, [&](int, int e, float z) { return __builtin_fmaf(z, cc, -sh[e / 4][e % 4]); });
            if (i % (4 * S::kNB) == 4 * S::kNB - 1) read_shift(i / (4 * S::kNB), shifts);
            if (i) s.template finished<Q>(i - 1, y);
          }
        });
        s.template finished<Q>(ALL - 1, y);
      }
      // a row whose target is among the wave's items (behind the last row all that is loaded is 0: a row of zeros,
      // whose product is 0 whatever P is)
      if (__builtin_expect(__any((t & ~kPlaces) == (int)own0), 0)) {
        uint32_t at = ax + 16 * s.h;
        asm volatile("" : "+v"(at));  // (one address and constants, not an address each)
        typedef int s32x4 __attribute__((ext_vector_type(4)));
        const int item = (int)own0 + s.lane % 32 * 4, row = (s0 + k) * kSweepStage + Q * 32 + s.lane;
        const uint32_t hits = (uint32_t)__ballot(row < n && (t & ~kPlaces) == (int)own0);  // (both halves' are alike)
        if (listed <= kRestList - 32) {
          if (s.lane < 32 && (hits >> s.lane & 1))
            *(CUTBCE_LDS uint32_t*)(size_t)(list + 16 + __builtin_amdgcn_mbcnt_lo(hits, listed) * 4) =
                (uint32_t)row * 128 + (uint32_t)(t & kPlaces) / 4;
          listed = uni(listed + __popc(hits));
        } else if (listed <= kRestList) {
          *(CUTBCE_LDS int*)(size_t)list = row - s.lane;
          listed = uni(listed + 2 * kRestList);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const s32x4 tr = *(CUTBCE_LDS const s32x4*)(size_t)(at + 256 + 32 * k);
          const f32x4 mine = *(CUTBCE_LDS const f32x4*)(size_t)(at + 512 + 32 * k);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t both = pack2(mine[2 * j], mine[2 * j + 1]);
#pragma unroll
            for (int b = 0; b < S::kNB; ++b) {
              uint32_t& p = s.p[Q][b][2 * k + j];
              p = tr[2 * j] == item + b * 128 ? (p & 0xffff0000u) | (both & 0xffffu) : p;
              p = tr[2 * j + 1] == item + b * 128 ? (p & 0xffffu) | (both & 0xffff0000u) : p;
            }
          }
        }
      }
      if constexpr (S::kPlain) s.last(Q);
    };
    s.settle();
    for (int k = 0; k < count; ++k) {
      landed_and_sync<(S::kAhead - 2) * S::kLoads>();
      step(std::integral_constant<int, 0>{}, k);
      step(std::integral_constant<int, 1>{}, k);
      s.move_on(S::step_of(k + 1), S::step_of(k));
      s.settle();
    }
    if constexpr (!S::kPlain) s.last(1);
    wait_and_sync<>();
    {
      static_assert(4 * kRests<DP> <= S::kLds, "");
      int lane = s.lane;
      asm volatile("" : "+v"(lane));  // (addresses are formed here, not kept through the loops above)
      int64_t last = (int64_t)(s0 + count) * kSweepStage, next;
      last = last < n ? last : n;
      next = listed > kRestList ? uni(*(CUTBCE_LDS const int*)(size_t)list) : last;
      for (int rests = listed > kRestList ? listed - 2 * kRestList : listed;;) {
        if (rests)
          multiply_rests<DP, S::kNB, DP <= 128 ? 2 : 1>(
              c, s.X, c.D, list + 16, rests, lane % 32, s.lds0 + s.wave * kRests<DP>, lane,
              [&](int d, bf16x8 features, const u32x4* items) INLINED {
                s.settle();
#pragma unroll
                for (int b = 0; b < S::kNB; ++b)
                  s.acc[d][b] = S::M::mma(__builtin_bit_cast(u32x4, features), items[b], s.acc[d][b]);
              });
        if (next >= last) break;
        rests = list_rests(c, next, last, list + 16, lane,
                           [&](int t) { return (t & ~kPlaces) == (int)own0 ? (t & kPlaces) / 4 : -1; });
      }
    }
    const float f = whole ? *grad * fabsf(c.scale) : 1.f;
#pragma unroll
    for (int b = 0; b < S::kNB; ++b) {
      const int at = (b * 32 + s.lane % 32) * 4 + s.wave;
      const int64_t v = tile * S::kOwned + at;
      if (v >= c.V) continue;
      f32x16 o[S::NDB];
#pragma unroll
      for (int d = 0; d < S::NDB; ++d) o[d] = s.acc[d][b];
      const int64_t piece = blockIdx.x * 2 + place;
      if (whole) store_row<__bf16, S::NDB>(dE + v * c.D, o, f, c.D, s.lane);
      else store_row<float, S::NDB>(sums + (piece * S::kOwned + at) * c.D, o, f, c.D, s.lane);
    }
  }
}

// What is left when the sweep is done, four features a lane. The first `pieces` workgroups: the tiles that were
// shared, each by the first workgroup of its parts but one. The others: dH of all rows from saved's, zeros for those
// left out.
__global__ __launch_bounds__(256) void k_ce_finish(Ce c, const float* __restrict__ sums, int64_t spread, int pieces,
                                                   const float* __restrict__ grad, __bf16* __restrict__ dH,
                                                   __bf16* __restrict__ dE) {
  typedef __bf16 V4 __attribute__((ext_vector_type(4)));
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  V4* to;
  float f;
  if ((int)blockIdx.x >= pieces) {
    const int64_t x = ((int64_t)(blockIdx.x - pieces) * 256 + threadIdx.x) * 4;
    if (x >= c.R * c.D) return;
    const int64_t r = x / c.D;
    const int i = at<int32_t>(c.saved, c.at.place)[r];
    if (i >= 0) s = *(const f32x4*)(at<float>(c.saved, c.at.dh) + (int64_t)i * c.D + (x - r * c.D));
    f = *grad * c.scale, to = (V4*)(dH + x);
    if (i < 0) f = 0.f;
  } else {
    const Line line(at<CeHead>(c.saved, c.at.head)->n, c.V, c.D);
    const int parts = items_grid(c.D) - 1;
    const int part = blockIdx.x % parts + 1;  // of the tile's second piece
    if (part >= line.parts) return;
    const int64_t cut = line.begin(part), at_tile = cut / line.stages, x0 = at_tile * line.stages;
    const int owned = sweep_rows(c.D);
    const int64_t tile = at_tile * spread % cdiv(c.V, owned);
    const int64_t before = line.begin(part - 1);
    if (cut == x0 || before > x0) return;  // cut at a tile's end, or not the tile's first cut
    const int64_t v0 = tile * owned, rows = c.V - v0 < owned ? c.V - v0 : owned;
    const int64_t x = ((int64_t)(blockIdx.x / parts) * 256 + threadIdx.x) * 4;
    if (x >= rows * c.D) return;
    const int64_t piece = (int64_t)owned * c.D;
    s = *(const f32x4*)(sums + ((int64_t)(part - 1) * 2 + (before == x0 ? 0 : 1)) * piece + x);
    for (int p = part; p < line.parts && line.begin(p) < x0 + line.stages; ++p)
      s += *(const f32x4*)(sums + (int64_t)p * 2 * piece + x);
    f = *grad * fabsf(c.scale), to = (V4*)(dE + v0 * c.D + x);
  }
  V4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = (__bf16)(s[j] * f);
  *to = y;
}

// The line's tiles are taken in steps of this many, a golden section of them with no common factor: neighbouring items,
// often those that are targets most, go to different workgroups. (One with the first 13 of 3,422 tiles of items by
// popularity took 30% longer than the others.)
int64_t spread_of(int64_t tiles) {
  int64_t m = tiles * 618 / 1000;
  if (m < 1) return 1;
  for (;; ++m) {
    int64_t a = m, b = tiles;
    while (b) {
      const int64_t t = a % b;
      a = b, b = t;
    }
    if (a == 1) return m;
  }
}

struct RowsPlan {
  size_t part, sums, off, bytes;
};
RowsPlan rows_plan(int64_t R, int D, bool grad) {
  // shares x rows are at most the units of all turns, or a share of each row
  const int64_t some = (int64_t)kSweepUnits * (R < sweep_rows(D) ? R : sweep_rows(D));
  const int64_t slots = some > R ? some : R;
  RowsPlan p;
  size_t b = 0;
  p.part = b, b += up(slots * 8, 256);
  p.sums = b, b += grad ? up(slots * D * 4, 256) : 0;
  const int64_t tiles = cdiv(R, sweep_rows(D));
  p.off = b, b += up((tiles > kSweepUnits ? tiles : kSweepUnits) * 4, 256);
  p.bytes = b;
  return p;
}

// Rows from which on they are joined a wave each (by a workgroup and by a wave: 2,048 rows, 100,000 x 64 9.6 and 9.5
// us, 5,120 15.7 and 10.0, 15,503 rows, 1,613 x 200 42 and 17).
constexpr int64_t kManyRows = 2048;

template <int DP, bool GRAD> hipError_t rows_t(const Ce& c, char* ws, const float* zt, float* row_loss, float* each,
                                               hipStream_t st) {
  using S = Sweep<DP, false, GRAD>;
  const RowsPlan p = rows_plan(c.R, c.D, GRAD);
  hipError_t e = allow_lds<k_ce_sweep_rows<DP, GRAD, false>>(S::kLds);
  if (e == hipSuccess) e = allow_lds<k_ce_sweep_rows<DP, GRAD, true>>(S::kLds);
  if (e != hipSuccess) return e;
  float2* part = (float2*)(ws + p.part);
  float* sums = (float*)(ws + p.sums);
  int* off = (int*)(ws + p.off);
  k_ce_sweep_rows<DP, GRAD, false><<<sweep_grid(c.D), 256, S::kLds, st>>>(c, part, sums, off);
  k_ce_sweep_rows<DP, GRAD, true><<<sweep_grid(c.D), 256, S::kLds, st>>>(c, part, sums, off);
  if (GRAD) {
    const unsigned waves = (unsigned)cdiv(c.R, 4);
    if (c.R >= kManyRows) k_ce_sweep_join<true><<<waves, 256, 0, st>>>(c, part, sums, zt, row_loss, each);
    else k_ce_sweep_join<false><<<(unsigned)c.R, 256, 0, st>>>(c, part, sums, zt, row_loss, each);
  }
  return hipGetLastError();
}

template <int DP>
hipError_t items_t(const Ce& c, float* sums, const float* grad, int64_t far, __bf16* dE, hipStream_t st) {
  constexpr int kLds = Sweep<DP, true, true>::kLds + 4 * kListBytes;
  static_assert(kLds * kWaves<DP, true> <= 160 * 1024, "");
  const hipError_t e = allow_lds<k_ce_sweep_items<DP>>(kLds);
  if (e != hipSuccess) return e;
  k_ce_sweep_items<DP><<<items_grid(c.D), 256, kLds, st>>>(c, grad, far, dE, sums);
  return hipGetLastError();
}

}  // namespace

bool ce_swept(int D, int dtype) { return dtype == 1 && D <= 256; }

size_t ce_rows_bytes(int64_t R, int D, bool grad) { return rows_plan(R, D, grad).bytes; }
hipError_t launch_ce_rows(const Ce& c, char* ws, bool grad, const float* zt, float* row_loss, float* each,
                          hipStream_t st) {
  auto by = [&](auto width) {
    constexpr int DP = decltype(width)::value;
    return grad ? rows_t<DP, true>(c, ws, zt, row_loss, each, st) : rows_t<DP, false>(c, ws, zt, row_loss, each, st);
  };
  return c.D <= 64    ? by(std::integral_constant<int, 64>{})
         : c.D <= 128 ? by(std::integral_constant<int, 128>{})
                      : by(std::integral_constant<int, 256>{});
}
size_t ce_items_bytes(int D) { return (size_t)items_grid(D) * 2 * sweep_rows(D) * D * 4; }
hipError_t launch_ce_items(const Ce& c, char* ws, const float* grad, void* dH, void* dE, hipStream_t st) {
  const int64_t far = spread_of(cdiv(c.V, sweep_rows(c.D)));
  float* sums = (float*)ws;
  if (dE) {
    const hipError_t e = c.D <= 64    ? items_t<64>(c, sums, grad, far, (__bf16*)dE, st)
                         : c.D <= 128 ? items_t<128>(c, sums, grad, far, (__bf16*)dE, st)
                                      : items_t<256>(c, sums, grad, far, (__bf16*)dE, st);
    if (e != hipSuccess) return e;
  }
  const int pieces = dE ? (items_grid(c.D) - 1) * (int)cdiv((int64_t)sweep_rows(c.D) * c.D, 1024) : 0;
  const int64_t blocks = pieces + (dH ? cdiv(c.R * c.D, 1024) : 0);
  if (blocks) k_ce_finish<<<(unsigned)blocks, 256, 0, st>>>(c, sums, far, pieces, grad, (__bf16*)dH, (__bf16*)dE);
  return hipGetLastError();
}

}  // namespace cutbce
