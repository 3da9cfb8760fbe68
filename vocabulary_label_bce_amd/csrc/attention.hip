// Causal attention over packed sequences or a key/value cache, with grouped heads, and its gradients.
//
//   out = softmax(s q k^T) v, row t of a sequence of n rows and m keys seeing the keys j <= t + m - n
//   P = exp(s q k^T - lse), dP = dO v^T, delta = rowsum(dO * out), dS = P * (dP - delta)
//   dv = P^T dO, dk = s dS^T q, dq = s dS k, dk and dv summed over the query heads that share them
//
// All products run on 32x32 matrix instructions with one side's rows as the columns of the result, so that a lane
// holds values of one row (or key) only: lane l has column l % 32, and of the rows acc_row(i, l / 32), i < 16. The
// forward and dq form S^T = K Q^T: a row's maximum and sum are the lane's own, joined with lane l ^ 32, and P^T (or
// dS^T) is the second product's B operand as it stands, with the keys in the order acc_row. dk and dv form S = Q K^T
// likewise with the keys as columns. The second product's A operand is the transpose of a tile that is in LDS
// row by row: for 16-bit elements the LDS transpose read delivers it, for float32 a plain read does.
//
// Tiles go from memory to LDS by direct buffer loads. A tile's rows past the sequence's end and columns past
// head_dim lie outside the buffer's range and arrive as zeros. The 16-byte chunks of a row are permuted by the
// row (swz) so that both the row-wise and the transposed reads spread over the LDS banks.
#include <atomic>
#include <type_traits>

#include "encoder.h"

namespace cutbce {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
#define CUTBCE_LDS __attribute__((address_space(3)))

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kRows = 128;  // rows (or keys) of a workgroup: four waves of 32
constexpr float kLazy = 8.f;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

__host__ __device__ constexpr inline int acc_row(int i, int h) { return (i / 4) * 8 + h * 4 + (i % 4); }

__device__ inline int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline int64_t uni64(int64_t x) {
  return (int64_t)(((uint64_t)(uint32_t)uni((int)(x >> 32)) << 32) | (uint32_t)uni((int)x));
}
__device__ inline float other_half(float x) {  // the value of lane l ^ 32
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}
__device__ inline float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// A tile of rows in LDS: DH features padded to a power of two, CPR 16-byte chunks a row, chunk c of row r at
// c ^ swz(r).
template <typename T, int DH> struct Tile {
  static constexpr int kEsz = sizeof(T);
  static constexpr int kRowB = (DH <= 32 ? 32 : (DH <= 64 ? 64 : 128)) * kEsz;
  static constexpr int kCPR = kRowB / 16;
  static constexpr int kNT = DH * kEsz / 32;  // pairs of chunks: k-steps of a product over the features
  static constexpr int kNDB = DH / 32;        // 32-wide blocks of features
  // LDS has 64 banks, 256 bytes: a row-wise read takes one chunk of 16 rows at a time, a transpose read four chunks of
  // four rows (from a multiple of 4), a float32 transposed read 128 bytes of rows r and r + 4. The row's bits are dealt
  // to the chunk's so that each of these covers the banks once. (Dealt for 32 banks the transpose reads took twice as
  // long.)
  __device__ static inline int swz(int r) {
    if constexpr (kCPR == 4) return (r >> 2) & 3;
    else if constexpr (kCPR == 8) return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
    else if constexpr (kEsz == 2) return (r & 3) << 2 | ((r >> 2) & 3);
    else return ((r >> 2) & 1) << 3 | ((r >> 3) & 1) << 2 | (r & 3);
  }
};

// Direct loads from memory to LDS, 16 or 4 bytes a lane from byte `voff` of the buffer to LDS byte `dst` (uniform) +
// lane * 16 (4); zeros where the buffer ends. As instructions of their own, not as the builtin (which k_attn_few uses
// for bf16, where it took 80 us and these 84): before a transpose read the compiler waits for every load to LDS that it
// knows to be in flight, those of the next stages as well. Nothing is returned in registers; the kernels wait for these
// loads themselves, before the stage is read and before the workgroup ends, and for the reads of a stage before it is
// loaded over: the compiler may move LDS reads past these loads, but not past those waits. The s_nop covers the wait
// states between a scalar register's write by a vector instruction (v_readfirstlane) or m0's and its use here.
__device__ inline u32x4 buffer_of(const void* base, int bytes) {  // uniform
  const uint64_t at = (uint64_t)base;
  return u32x4{(uint32_t)uni((int)at), (uint32_t)uni((int)(at >> 32)) & 0xffffu, (uint32_t)uni(bytes), 0x00020000u};
}
__device__ inline void load_lds16(u32x4 buffer, int voff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(uni(dst)), "v"(voff), "s"(buffer) : "m0");
}
__device__ inline void load_lds4(u32x4 buffer, int voff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(uni(dst)), "v"(voff), "s"(buffer) : "m0");
}

// One workgroup's (or wave's) loads of NR rows into LDS: NL lanes, 16 bytes each per instruction.
template <typename T, int DH, int NR, int NL> struct Dma {
  using Ti = Tile<T, DH>;
  static constexpr int kChunks = NR * Ti::kCPR, kLanes = kChunks < NL ? kChunks : NL;  // whole waves load
  static constexpr int kRounds = kChunks / kLanes, kStep = kLanes / Ti::kCPR;            // rows per round
  static constexpr int kBytes = NR * Ti::kRowB;
  static_assert(kRounds * kStep == NR && kLanes % 64 == 0, "");
  bool on;
  int row, chunk, step;  // this lane's row offset in bytes and chunk in the first round; bytes from round to round
  __device__ inline void init(int lane, int64_t stride) {
    on = lane < kLanes;
    const int r = lane / Ti::kCPR;
    row = (int)(r * stride * Ti::kEsz);
    chunk = (lane % Ti::kCPR) ^ Ti::swz(r);
    step = (int)(stride * Ti::kEsz) * kStep;
  }
  // round q's rows are kStep q further on: swz is linear in the row's bits, and r < kStep
  __device__ inline int offset(int q, int dh) const {
    const int c = (chunk ^ Ti::swz(q * kStep)) * 16;
    return c < dh * Ti::kEsz ? row + c + q * step : (int)0x80000000u;
  }
  // the range of rows [0, rem) of `base`, and one round of its loads (for kernels that spread them)
  __device__ inline u32x4 range(const T* base, int64_t rem, int64_t stride, int dh) const {
    const int rows = (int)clamp64(rem, 0, NR);
    return buffer_of(base, rows > 0 ? (int)((rows - 1) * stride + dh) * Ti::kEsz : 0);
  }
  __device__ inline void round(int q, u32x4 range, int dh, uint32_t dst) const {
    if (kLanes < NL && !on) return;
    load_lds16(range, offset(q, dh), dst + q * kLanes * 16);
  }
  // rows [0, rem) of `base` (uniform; rem may be <= 0 or > NR) to LDS byte `dst` (uniform: the wave's first kilobyte)
  __device__ inline void load(const T* base, int64_t rem, int64_t stride, int dh, uint32_t dst) const {
    if (kLanes < NL && !on) return;
    const int rows = (int)clamp64(rem, 0, NR);
    const int bytes = rows > 0 ? (int)((rows - 1) * stride + dh) * Ti::kEsz : 0;
#if defined(__HIP_DEVICE_COMPILE__)  // (the host pass silently drops kernels that reach these builtins this way)
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, bytes, 0x00020000);
#pragma unroll
    for (int q = 0; q < kRounds; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (CUTBCE_LDS void*)(size_t)(dst + q * kLanes * 16), 16, offset(q, dh),
                                               0, 0, 0);
#endif
  }
};

// (x, y) of 32 rows as 32 x's and 32 y's to LDS byte `dst` (uniform); zeros behind `rows`.
__device__ inline void load_pairs(const float2* base, int64_t rows, uint32_t dst, int lane) {
  load_lds4(buffer_of(base, (int)clamp64(rows, 0, 32) * 8), (lane % 32) * 8 + (lane / 32) * 4, dst);
}

__device__ inline u32x4 lds16(uint32_t at) { return *(CUTBCE_LDS const u32x4*)(size_t)at; }

template <typename T> struct Mma;

template <> struct Mma<__bf16> {
  struct P { bf16x8 g[2]; };  // a 32x32 result as the second product's B operand
  __device__ static inline f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  __device__ static inline u32x4 negate(u32x4 x) { return x ^ 0x80008000u; }
  __device__ static inline P pack(const f32x16& x) {  // rounds to nearest even
    P p;
#pragma unroll
    for (int i = 0; i < 16; ++i) p.g[i / 8][i % 8] = (__bf16)x[i];
    return p;
  }
  // acc += X^T P, X 32 rows of a tile: kSlotsPerBlock matrix instructions for each block of features, the blocks in
  // turn, each with an operand of its own. An operand's address is the lane's base for the tile with the slot's chunk
  // bits flipped and its rows added, both constants: the bases are formed for each tile, so that no register holds an
  // address from one tile to the next (tiles start at a multiple of their row's size).
  typedef bf16x8 A;
  static constexpr int kSlotsPerBlock = 2;
  template <int DH> __device__ static inline uint32_t base_t(uint32_t at, int lane) {
    using Ti = Tile<__bf16, DH>;
    const int s = lane % 16, row = 4 * (lane / 32) + s / 4;
    return at + row * Ti::kRowB + ((2 * ((lane / 16) & 1) + ((s & 3) >> 1)) ^ Ti::swz(row)) * 16 + (s & 1) * 8;
  }
  template <int DH> __device__ static inline A load_t(int slot, uint32_t base) {
    using Ti = Tile<__bf16, DH>;
    const int g = slot / Ti::kNDB, db = slot % Ti::kNDB;
    s16x4 x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      x[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CUTBCE_LDS s16x4*)(size_t)(
          (base ^ ((db * 4) ^ Ti::swz(16 * g + 8 * e)) * 16) + (16 * g + 8 * e) * Ti::kRowB));
    return __builtin_bit_cast(A, (s16x8)__builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
  }
  template <int NDB> __device__ static inline void slot_t(f32x16* acc, int slot, A a, const P& p) {
    acc[slot % NDB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, p.g[slot / NDB], acc[slot % NDB], 0, 0, 0);
  }
};

template <> struct Mma<float> {
  typedef f32x16 P;
  __device__ static inline f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], c, 0, 0, 0);
    return c;
  }
  __device__ static inline u32x4 negate(u32x4 x) { return x ^ 0x80000000u; }
  __device__ static inline P pack(const f32x16& x) { return x; }
  typedef float A;
  static constexpr int kSlotsPerBlock = 16;
  template <int DH> __device__ static inline uint32_t base_t(uint32_t at, int lane) {
    using Ti = Tile<float, DH>;
    const int n = lane % 32, row = 4 * (lane / 32);
    return at + row * Ti::kRowB + ((n / 4) ^ Ti::swz(row)) * 16 + (n % 4) * 4;
  }
  template <int DH> __device__ static inline A load_t(int slot, uint32_t base) {
    using Ti = Tile<float, DH>;
    const int row = acc_row(slot / Ti::kNDB, 0);
    return *(CUTBCE_LDS const float*)(size_t)((base ^ (((slot % Ti::kNDB) * 8) ^ Ti::swz(row)) * 16) + row * Ti::kRowB);
  }
  template <int NDB> __device__ static inline void slot_t(f32x16* acc, int slot, A a, const P& p) {
    acc[slot % NDB] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p[slot / NDB], acc[slot % NDB], 0, 0, 0);
  }
};

// acc += X^T P, scheduled by the compiler: X the 32 rows at `at`.
template <typename T, int DH>
__device__ inline void product_t(f32x16* acc, const typename Mma<T>::P& p, uint32_t at, int lane) {
  constexpr int NDB = Tile<T, DH>::kNDB;
  const uint32_t base = Mma<T>::template base_t<DH>(at, lane);
#pragma unroll
  for (int k = 0; k < Mma<T>::kSlotsPerBlock * NDB; ++k)
    Mma<T>::template slot_t<NDB>(acc, k, Mma<T>::template load_t<DH>(k, base), p);
}

// acc += X^T P with what the rounding of P to 16 bits leaves over, as a second part: twice the matrix instructions,
// each pair with one operand of X.
template <typename T, int DH> __device__ inline void product_t_exact(f32x16* acc, f32x16 x, uint32_t at, int lane) {
  if constexpr (sizeof(T) == 4) {
    product_t<T, DH>(acc, Mma<T>::pack(x), at, lane);
  } else {
    constexpr int NDB = Tile<T, DH>::kNDB;
    const typename Mma<T>::P p = Mma<T>::pack(x);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] -= to_f32(p.g[i / 8][i % 8]);
    const typename Mma<T>::P rest = Mma<T>::pack(x);
    const uint32_t base = Mma<T>::template base_t<DH>(at, lane);
#pragma unroll
    for (int k = 0; k < Mma<T>::kSlotsPerBlock * NDB; ++k) {
      const typename Mma<T>::A t = Mma<T>::template load_t<DH>(k, base);
      Mma<T>::template slot_t<NDB>(acc, k, t, p);
      Mma<T>::template slot_t<NDB>(acc, k, t, rest);
    }
  }
}

// The tile's operand of k-step t: the 32 rows from `at`, through the lane's base as above.
template <typename T, int DH> __device__ inline uint32_t base_row(uint32_t at, int lane) {
  using Ti = Tile<T, DH>;
  const int r = lane % 32;
  return at + r * Ti::kRowB + ((lane / 32) ^ Ti::swz(r)) * 16;
}
__device__ inline u32x4 load_row(uint32_t base, int t) { return lds16(base ^ (2 * t * 16)); }

// 32 rows of a tile times the own operand: the result's rows are the tile's, its columns the own rows.
template <typename T, int DH>
__device__ inline f32x16 product(uint32_t at, const u32x4* own, int lane) {
  using Ti = Tile<T, DH>;
  const uint32_t base = base_row<T, DH>(at, lane);
  f32x16 s = {};
#pragma unroll
  for (int t = 0; t < Ti::kNT; ++t) s = Mma<T>::mma(load_row(base, t), own[t], s);
  return s;
}

// Products with their order pinned in 16-bit elements, for kernels whose waves run in step: a product's matrix
// instructions are interleaved with the LDS reads of the operands that come after it. (Left alone, the compiler reads
// each operand right before its use and waits for it.)
template <typename T> __device__ inline void pin() {
  if constexpr (sizeof(T) == 2) __builtin_amdgcn_sched_barrier(0);
}
// f(e) for slot k's share of n things in `slots` slots
template <typename F> __device__ inline void spread(int k, int slots, int n, F f) {
#pragma unroll
  for (int e = n * k / slots; e < n * (k + 1) / slots; ++e) f(e);
}
template <typename T, int DH> struct Ahead {
  static constexpr int NT = Tile<T, DH>::kNT, NDB = Tile<T, DH>::kNDB, S = Mma<T>::kSlotsPerBlock * NDB;
  u32x4 x[NT];              // 32 rows of a tile
  typename Mma<T>::A t[S];  // 32 rows of a tile, transposed
  // (bases of the lane: rows_at and cols_at of a tile)
  __device__ static inline uint32_t rows_at(uint32_t at, int lane) { return base_row<T, DH>(at, lane); }
  __device__ static inline uint32_t cols_at(uint32_t at, int lane) { return Mma<T>::template base_t<DH>(at, lane); }
  __device__ inline void row(int k, uint32_t base) { x[k] = load_row(base, k); }
  __device__ inline void col(int e, uint32_t base) { t[e] = Mma<T>::template load_t<DH>(e, base); }
  __device__ inline void rows(uint32_t base) {
#pragma unroll
    for (int k = 0; k < NT; ++k) row(k, base);
  }
  // x times the own operand; work(k) after the k-th of NT steps, when x[k] is free
  template <typename F> __device__ inline f32x16 product(const u32x4* own, F work) {
    f32x16 s = {};
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      s = Mma<T>::mma(x[k], own[k], s);
      work(k);
      pin<T>();
    }
    return s;
  }
  // acc += t p; work(e) after the e-th of S steps, when t[e] is free
  template <typename F> __device__ inline void product_t(f32x16* acc, const typename Mma<T>::P& p, F work) {
#pragma unroll
    for (int e = 0; e < S; ++e) {
      Mma<T>::template slot_t<NDB>(acc, e, t[e], p);
      work(e);
      pin<T>();
    }
  }
};

// The own operand: lane l has the chunks 2t + l / 32 of one row (zeros past head_dim, or where !live).
template <typename T, int DH> __device__ inline void load_own(u32x4* own, const T* row, bool live, int dh, int lane) {
  using Ti = Tile<T, DH>;
  const int h = lane / 32;
#pragma unroll
  for (int t = 0; t < Ti::kNT; ++t) {
    const int c = 2 * t + h;
    u32x4 x = {0, 0, 0, 0};
    if (live && c * 16 < dh * Ti::kEsz) x = *(const u32x4*)((const char*)row + c * 16);
    own[t] = x;
  }
}

// A transposed result (lane: one row, the features 32 db + acc_row) times f, to a row of dh elements.
template <typename T, int NDB> __device__ inline void store_row(T* row, const f32x16* acc, float f, int dh, int lane) {
  const int h = lane / 32;
#pragma unroll
  for (int db = 0; db < NDB; ++db)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = db * 32 + 8 * k + 4 * h;
      if (d < dh) {
        typedef T V4 __attribute__((ext_vector_type(4)));
        V4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (T)(acc[db][4 * k + j] * f);
        *(V4*)(row + d) = v;
      }
    }
}

// Work units: tiles of M rows, units_of(rows, seqs, M) numbers for them.
//
// Up to 63 sequences: the units are numbered by the tiles left from them to one end of their sequence, most first
// (ENDS: a tile counts those before it, for kernels whose later tiles see more; else those behind it), so that the
// workgroups that take longest start first whatever the sequences' order. A lane has a sequence's number of tiles T;
// the level of unit u is the l with sum max(0, T - l - 1) <= u < sum max(0, T - l). At 4 x 8192 the forward, whose
// longest workgroup has as many steps as each of the 512 places gets in all, took 313 us with the sequences one after
// another and 275 so.
//
// More sequences than a wave has lanes for: sequence b's tiles start at unit start(b) / M + b, which leaves room for
// each of them (a range of n rows spans at least ceil(n / M) of these numbers), so that no running total is needed; the
// lanes look at 64 sequences at a time.
struct Unit {
  SeqRange s;
  int tile;  // tile of the sequence; may lie behind its end
};
__device__ inline int64_t start_of(const int32_t* cu, int64_t pitch, int64_t rows, int b) {
  return cu ? clamp64(cu[b], 0, rows) : b * pitch;
}
template <int M, bool ENDS>
__device__ inline Unit find_unit(const Attn& a, const int32_t* cu, int64_t pitch, int64_t rows, int64_t unit) {
  const int lane = threadIdx.x % 64;
  Unit u;
  int seq;
  if (a.seqs < 64) {
    int64_t from = 0, to = 0;
    if (lane <= a.seqs) {
      from = start_of(cu, pitch, rows, lane);
      to = lane == a.seqs ? rows : start_of(cu, pitch, rows, lane + 1);
    }
    const int T = to > from ? (int)((to - from + M - 1) / M) : 0;
    auto at_level = [&](int l) {  // tiles that have at least l others on the counted side
      int x = T > l ? T - l : 0;
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
      return x;
    };
    int lo = 0, hi = T;  // the level is in [lo, hi)
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const int x = __shfl_xor(hi, o, 64);
      hi = hi > x ? hi : x;
    }
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (at_level(mid) > unit) lo = mid; else hi = mid;
    }
    int r = (int)clamp64(unit - at_level(lo + 1), 0, 1 << 30);
    uint64_t m = __ballot(T > lo);
    while (r > 0 && m) m &= m - 1, --r;
    seq = m ? __builtin_ctzll(m) : a.seqs;
    const int n = __shfl(T, seq, 64);
    u.tile = m ? (ENDS ? lo : n - 1 - lo) : 1 << 30;  // (no m: a number beyond the last unit)
  } else {
    int lo = 0, cnt = a.seqs + 1;
    while (cnt > 1) {
      const int step = (cnt + 63) / 64, at = lane * step;
      const bool ok = at < cnt && start_of(cu, pitch, rows, lo + at) / M + lo + at <= unit;
      const uint64_t m = __ballot(ok);
      const int n = m ? 63 - __builtin_clzll(m) : 0;
      lo += n * step;
      cnt = cnt - n * step < step ? cnt - n * step : step;
    }
    seq = lo;
    u.tile = (int)clamp64(unit - (start_of(cu, pitch, rows, lo) / M + lo), 0, 1 << 30);
  }
  u.tile = uni(u.tile);
  const SeqRange s = seq_range(a, uni(seq));
  u.s.q0 = uni64(s.q0), u.s.k0 = uni64(s.k0), u.s.kb = uni64(s.kb), u.s.vb = uni64(s.vb);
  u.s.n = uni(s.n), u.s.m = uni(s.m), u.s.cap = uni(s.cap);
  return u;
}
int64_t units_of(int64_t rows, int seqs, int m = kRows) { return rows / m + seqs + 1; }

// Keys that row t of the sequence sees.
__device__ inline int seen_by(const Attn& a, const SeqRange& s, int64_t t) {
  return a.causal ? (int)clamp64(t + s.m - s.n + 1, 0, s.m) : s.m;
}

// Waits until at most N of the wave's loads are in flight and its LDS accesses are done, then for the workgroup.
template <int N = 0> __device__ inline void wait_and_sync() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename T, int DH> constexpr int key_tile() { return sizeof(T) == 4 && DH > 64 ? 32 : 64; }
// LDS stages of the forward and dq: two of 32 KB, or four smaller ones, so that a short sequence's keys are all on
// their way at once.
template <typename T, int DH> constexpr int key_stages() { return key_tile<T, DH>() * Tile<T, DH>::kRowB > 8192 ? 2 : 4; }

// Exponents are scale * log2 e * (q . k) less a row's reference R. In one fused step, x * c - R, they are off by R's
// own rounding, alike for the whole row: that cancels in the softmax, but it passes 128 from R = 2^31 on. So where a
// row's reference is beyond kBig the product is rounded first, as R was, and the largest exponent is 0 (up to there
// R's rounding is under 2^-11; ordinary scores are in the tens). And references are kept as R / 2 (c / 2 times the
// scores; a factor of 2 is exact): scale * (q . k) up to float32's largest value is 1.44 times that in base 2.
constexpr float kBig = 4096.f;  // of R / 2
__device__ inline float rounded_less(float x, float c, float r) {
#pragma clang fp contract(off)
  const float p = x * c;
  return p - r;
}
__device__ inline float rounded_product(float x, float c) {
#pragma clang fp contract(off)
  return x * c;
}

// Running softmax of one row per lane: `half` is R / 2, from the largest score so far or one not far below it.
struct Online {
  float half = -INFINITY, sum = 0.f;
};

// What the forward multiplies: q, negated for a negative scale and 0 for a scale of 0 (or one too small for c / 2), so
// that c / 2 = |scale| log2 e / 2 is above 0 and a masked score of -inf stays so.
template <typename T, int NT> __device__ inline float half_scale(float scale, u32x4* own) {
  const float ch = fabsf(scale) * (0.5f * kLog2e);
  if (scale < 0.f) {
#pragma unroll
    for (int i = 0; i < NT; ++i) own[i] = Mma<T>::negate(own[i]);
  }
  if (ch > 0.f) return ch;
#pragma unroll
  for (int i = 0; i < NT; ++i) own[i] = u32x4{0, 0, 0, 0};
  return 1.f;
}

// P from scores of NS 32-key blocks (row-wise, ch = scale * log2 e / 2 > 0); rescales the output when a row's maximum
// has grown by more than a factor of 2^kLazy since it was last used (the exponentials stay below 2^kLazy until then).
template <int NS, int NDB> __device__ inline void softmax_step(f32x16* s, float ch, Online& st, f32x16* o) {
  float mx = s[0][0];
#pragma unroll
  for (int b = 0; b < NS; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
  mx = fmaxf(mx, other_half(mx));
  mx = rounded_product(mx, ch);
  if (__any(mx > st.half + 0.5f * kLazy)) {
    const float nw = fmaxf(st.half, mx);
    const float f = st.half == -INFINITY ? 0.f : exp2_of(2.f * (st.half - nw));
    st.half = nw;
    st.sum *= f;
#pragma unroll
    for (int d = 0; d < NDB; ++d) o[d] *= f;
  }
  const float half = st.half == -INFINITY ? 0.f : st.half;
  float c = 2.f * ch, base = 2.f * half;
  if (__builtin_expect(__any(fabsf(half) > kBig), 0)) {
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = rounded_less(s[b][i], ch, half);
    c = 2.f, base = 0.f;
  }
#pragma unroll
  for (int b = 0; b < NS; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[b][i] = exp2_of(__builtin_fmaf(s[b][i], c, -base));
      st.sum += s[b][i];
    }
}

// (beyond kBig as the backward forms it again from a score, see big_exponent)
__device__ inline float finish_lse(float half, float sum, bool any) {
  if (!any) return -INFINITY;
  const float l = __builtin_amdgcn_logf(sum);
  return fabsf(half) > kBig ? rounded_product(half, 2.f * kLn2) + l * kLn2 : (2.f * half + l) * kLn2;
}

// The backward's exponent from lse where that is beyond kBigLse: rounded as the forward rounded it, so that a row's
// largest score gives log2 of what its sum left in lse, and never more than 0. (P is then off by 2^-24 |lse| of itself,
// lse's own rounding; from 2^27 on the sum is lost altogether: P = 1 at a row's largest score.)
constexpr float kBigLse = kBig * 2.f * kLn2;
__device__ inline float big_exponent(float x, float ch, float lse) {
  const float y = rounded_less(rounded_product(x, ch), 2.f * kLn2, lse) * kLog2e;
  return y > 0.f ? 0.f : y;
}

// Forward: a workgroup has 128 rows of one sequence and head, a wave 32 of them; the keys stream through LDS stages of
// KT keys, shared by the four waves. Two workgroups a CU (registers), so that a SIMD has a wave of each: one's softmax
// beside the other's products. 4 sequences of up to 8,192 rows, 8 heads over 2 of 128, bf16: 265 to 277 us (by the
// card), 930 to 970 TFLOP/s of the seen pairs; the matrix unit is busy 48% of the cycles and vector instructions issue
// in 41%, so a wave's chain of scores, softmax and product bounds it, and the tail of the longest sequences. 128
// sequences of up to 200 rows, 2 heads of 64: 11 us, latency (search, first tiles, up to four steps). In float32 one
// sequence of 2,048, 8 heads over 2 of 64, in 3 parts: 71 us and 5 for the join; its matrix instructions alone are 28.
//
// In bf16 the probabilities are rounded to bf16 for the product with the values: as an operand they have the precision
// that v has, each errs by at most 2^-8 of itself, with either sign, and out's error is 0.14 to 0.21% of its norm
// (0.17% is the rounding of out alone). A second part for what is left over, as in k_attn_few, would be half as many
// matrix instructions again as the forward has.
//
// SPLIT: `parts` workgroups for each tile of rows and head, with a share of its steps each (row_parts); they leave
// their sums and, for each row, its reference and the sum of its exponentials (-1 for a row that sees no key) for
// k_attn_fwd_join.
template <typename T, int DH, bool SPLIT>
__global__ __launch_bounds__(256, 2) void k_attn_fwd(Attn a, int parts, T* __restrict__ out, float* __restrict__ lse,
                                                     float* __restrict__ sums, float2* __restrict__ stats) {
  using Ti = Tile<T, DH>;
  constexpr int KT = key_tile<T, DH>(), NS = KT / 32, ST = key_stages<T, DH>();
  using Ld = Dma<T, DH, KT, 256>;
  extern __shared__ __align__(1024) char lds[];
  const uint32_t lds0 = uni((uint32_t)(size_t)(CUTBCE_LDS char*)lds);
  const int tid = threadIdx.x, wave = uni(tid / 64), lane = tid % 64;
  const unsigned part = SPLIT ? blockIdx.x % parts : 0, tile = SPLIT ? blockIdx.x / parts : blockIdx.x;
  const int h = tile % a.hq;
  const Unit u = find_unit<kRows, true>(a, a.cu_q, a.q_pitch, a.q_rows, tile / a.hq);
  const SeqRange& s = u.s;
  const int64_t r0 = (int64_t)u.tile * kRows;  // first row of the workgroup in its sequence
  if (r0 >= s.n) return;
  const int64_t t = r0 + wave * 32 + lane % 32;
  const bool live = t < s.n;
  const T* q = (const T*)a.q + (s.q0 + t) * a.q_rs + h * a.q_hs;
  u32x4 qo[Ti::kNT];
  load_own<T, DH>(qo, q, live, a.dh, lane);
  const float ch = half_scale<T, Ti::kNT>(a.scale, qo);
  const T* k = (const T*)a.k + s.kb + (h / a.group) * a.k_hs;
  const T* v = (const T*)a.v + s.vb + (h / a.group) * a.v_hs;
  const int mine = seen_by(a, s, t);                                     // keys of the lane's row
  const int wave_lo = seen_by(a, s, r0 + wave * 32);                     // fewest and most of the wave's rows
  const int wave_hi = r0 + wave * 32 < s.n ? seen_by(a, s, clamp64(r0 + wave * 32 + 31, 0, s.n - 1)) : 0;
  const int total = (seen_by(a, s, clamp64(r0 + kRows - 1, 0, s.n - 1)) + KT - 1) / KT;
  const int from = SPLIT ? (int)((int64_t)total * part / parts) : 0;
  const int steps = SPLIT ? (int)((int64_t)total * (part + 1) / parts) : total;  // this part's: from .. steps - 1
  Ld lk, lv;
  lk.init(tid, a.k_rs);
  lv.init(tid, a.v_rs);
  const uint32_t dst = lds0 + wave * 1024;
  u32x4 rk = {}, rv = {};
  uint32_t to = 0;
  auto prepare = [&](int i) {  // (beyond the last key the range is empty: zeros are loaded)
    const int64_t j = (int64_t)i * KT;
    rk = lk.range(k + j * a.k_rs, s.m - j, a.k_rs, a.dh);
    rv = lv.range(v + j * a.v_rs, s.m - j, a.v_rs, a.dh);
    to = dst + (i & (ST - 1)) * 2 * Ld::kBytes;
  };
  auto piece = [&](int q) {
    if (q < Ld::kRounds) lk.round(q, rk, a.dh, to);
    else lv.round(q - Ld::kRounds, rv, a.dh, to + Ld::kBytes);
  };
  constexpr int kPieces = 2 * Ld::kRounds;
  auto fetch = [&](int i) {
    prepare(i);
#pragma unroll
    for (int q = 0; q < kPieces; ++q) piece(q);
  };
  using Op = Ahead<T, DH>;
  f32x16 o[Ti::kNDB] = {};
  Online st;
  if (steps > from) {
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(from + i);
  }
  for (int i = from; i < steps; ++i) {
    wait_and_sync<(ST - 2) * kPieces>();  // tile i is there, tile i - 1 is done with
    const int j0 = i * KT;
    if (j0 >= wave_hi) {
      fetch(i + ST - 1);
      continue;
    }
    prepare(i + ST - 1);
    const uint32_t kt = lds0 + (i & (ST - 1)) * 2 * Ld::kBytes, vt = kt + Ld::kBytes;
    Op op;
    const uint32_t kr = Op::rows_at(kt, lane), vc = Op::cols_at(vt, lane);
    op.rows(kr);
    pin<T>();
    f32x16 x[NS];
#pragma unroll
    for (int b = 0; b < NS; ++b)
      x[b] = op.product(qo, [&](int n) {
        if (b + 1 < NS) op.row(n, kr + (b + 1) * 32 * Ti::kRowB);
        else spread(n, Op::NT, Op::S, [&](int e) { op.col(e, vc); });
        spread(b * Op::NT + n, NS * Op::NT, kPieces, piece);
      });
    if (j0 + KT > wave_lo) {
#pragma unroll
      for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (j0 + b * 32 + acc_row(e, lane / 32) >= mine) x[b][e] = -INFINITY;
    }
    softmax_step<NS, Ti::kNDB>(x, ch, st, o);
#pragma unroll
    for (int b = 0; b < NS; ++b)
      op.product_t(o, Mma<T>::pack(x[b]), [&](int e) {
        if (b + 1 < NS) op.col(e, vc + (b + 1) * 32 * Ti::kRowB);
      });
  }
  wait_and_sync<>();  // no load may reach LDS after the workgroup's end
  const float sum = st.sum + other_half(st.sum);
  if (live) {
    const int64_t at = (s.q0 + t) * a.hq + h;
    if constexpr (SPLIT) {
      const int64_t to = part * (a.q_rows * a.hq) + at;
      store_row<float, Ti::kNDB>(sums + to * a.dh, o, 1.f, a.dh, lane);
      if (lane < 32) stats[to] = make_float2(st.half, mine > 0 ? sum : -1.f);
    } else {
      store_row<T, Ti::kNDB>(out + at * a.dh, o, mine > 0 ? 1.f / sum : 0.f, a.dh, lane);
      if (lse && lane < 32) lse[at] = finish_lse(st.half, sum, mine > 0);
    }
  }
}

// Few tiles of rows leave CUs idle: the keys that a tile sees are then dealt to several workgroups, no more than two a
// CU in all, where a part gets 512 keys or more (256 in float32, whose products take longer) and there are three parts
// or more. One sequence of 4,096 rows, 1 head of 128, bf16, in 8 parts with the join: forward 74 -> 25 us, dq 98 ->
// 35; of 2,048, float32: 270 -> 47 and 406 -> 69. Two parts of 512 bf16 keys gain nothing over one workgroup (1,024
// rows, 2 heads of 64: 18 us): the join takes 4. Parts of half as many keys, forward and dq with their joins: bf16,
// 1,024 rows, 2 heads of 64 18.7 -> 14.5 and 23.9 -> 20.7 us, 2 x 1,500, 4 heads of 128 33.4 -> 25.8 and 43.6 -> 35.3,
// but 4 x 1,024, 4 heads of 64 (148 workgroups, 3 parts) 19.9 -> 20.0 and 25.1 -> 28.5; float32, 700 rows, 2 heads of
// 64 52 -> 24 and 74 -> 31, 4 x 500, 4 heads of 128 75 -> 41 and 111 -> 59. So these bounds are on the safe side.
int row_parts(const Attn& a) {
  const int64_t wgs = (a.q_rows / kRows + a.seqs + 1) * a.hq, most = a.k_pitch / (a.dtype == 1 ? 512 : 256);
  int64_t p = 512 / wgs;
  if (p > most) p = most;
  return (int)(most < 3 || p < 1 ? 1 : p);
}

// The parts' results of `rows` rows and heads joined in their order: 32 lanes a row, four features each.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_fwd_join(int parts, int64_t rows, int dh, const float* __restrict__ sums,
                                                       const float2* __restrict__ stats, T* __restrict__ out,
                                                       float* __restrict__ lse) {
  const int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int d = threadIdx.x % 32 * 4;
  if (r >= rows || d >= dh) return;
  const bool any = stats[r].y >= 0.f || stats[r].y != stats[r].y;
  float mx = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) mx = fmaxf(mx, stats[p * rows + r].x);
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float2 t = stats[p * rows + r];
    const float f = t.x == -INFINITY ? 0.f : exp2_of(2.f * (t.x - mx));
    sum += f * t.y;
    x += f * *(const f32x4*)(sums + (p * rows + r) * dh + d);
  }
  typedef T V4 __attribute__((ext_vector_type(4)));
  V4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = (T)(x[j] * (any ? 1.f / sum : 0.f));
  *(V4*)(out + r * dh + d) = y;
  if (lse && d == 0) lse[r] = finish_lse(mx, sum, any);
}


// dq, and the rows' (lse in base 2, delta) for dk and dv: the forward's layout and loop. At the forward's sizes 367 to
// 383 us (matrix unit busy 53%, vector issue 42%), 17 us, and in float32 103 us and 5 for the join. delta is needed
// from the first key on. dO . out with the rounded out is off by out's rounding, which few keys leave as large as dS
// itself (bf16: dq off by 0.33% of its norm at 4 keys, 0.28% at 16, 0.25% from 256 on; 0.23% is the rounding of dS and
// dq). So where a workgroup's keys fit into the LDS stages all at once (256 keys, 128 at head_dim over 64), a first
// pass over them there sums P dP in float32 instead: dq off by 0.23%, 14 -> 16 us at 128 sequences of up to 200. The
// workgroups with more keys take dO . out (their rows then add little: 0.24% at any length); what it is off by is the
// sum of a row's dS in float32, and dk gets it added.
//
// SPLIT: `parts` workgroups for each tile of rows and head, as in the forward; they leave their sums (of dS in off) for
// k_attn_dq_join. The first one takes all of the keys where they fit into LDS.
template <typename T, int DH, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(T) == 4 && DH > 64 ? 1 : 2) void k_attn_dq(
    Attn a, int parts, const T* __restrict__ dout, const T* __restrict__ out, const float* __restrict__ lse,
    T* __restrict__ dq, float2* __restrict__ stat, float* __restrict__ sums, float* __restrict__ off) {
  using Ti = Tile<T, DH>;
  constexpr int KT = key_tile<T, DH>(), NS = KT / 32, ST = key_stages<T, DH>();
  using Ld = Dma<T, DH, KT, 256>;
  extern __shared__ __align__(1024) char lds[];
  const uint32_t lds0 = uni((uint32_t)(size_t)(CUTBCE_LDS char*)lds);
  const int tid = threadIdx.x, wave = uni(tid / 64), lane = tid % 64;
  const unsigned part = SPLIT ? blockIdx.x % parts : 0, tile = SPLIT ? blockIdx.x / parts : blockIdx.x;
  const int h = tile % a.hq;
  const Unit u = find_unit<kRows, true>(a, a.cu_q, a.q_pitch, a.q_rows, tile / a.hq);
  const SeqRange& s = u.s;
  const int64_t r0 = (int64_t)u.tile * kRows;
  if (r0 >= s.n) return;
  const int64_t t = r0 + wave * 32 + lane % 32;
  const bool live = t < s.n;
  const int64_t at = (s.q0 + t) * a.hq + h;
  u32x4 qo[Ti::kNT], go[Ti::kNT];
  load_own<T, DH>(qo, (const T*)a.q + (s.q0 + t) * a.q_rs + h * a.q_hs, live, a.dh, lane);
  load_own<T, DH>(go, dout + at * a.dh, live, a.dh, lane);
  const int mine = live ? seen_by(a, s, t) : 0;
  // a row that sees no key has lse = -inf; +inf makes its probabilities 0
  const float ln = mine > 0 ? lse[at] : INFINITY;
  const bool big = fabsf(ln) > kBigLse && fabsf(ln) < INFINITY, any_big = __any(big);
  const float L0 = big ? ln : ln * kLog2e;
  float off_by = 0.f;  // sum dS
  const float c0 = a.scale * kLog2e, ch = a.scale * (0.5f * kLog2e);
  const float c = any_big ? 1.f : c0, L = any_big ? 0.f : L0;
  auto look = [&](f32x16& x) {  // scores that are to be c x - L from here on
    if (__builtin_expect(any_big, 0)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = big ? big_exponent(x[e], ch, L0) : __builtin_fmaf(x[e], c0, -L0);
    }
  };
  const T* k = (const T*)a.k + s.kb + (h / a.group) * a.k_hs;
  const T* v = (const T*)a.v + s.vb + (h / a.group) * a.v_hs;
  const int wave_lo = seen_by(a, s, r0 + wave * 32);
  const int wave_hi = r0 + wave * 32 < s.n ? seen_by(a, s, clamp64(r0 + wave * 32 + 31, 0, s.n - 1)) : 0;
  const int total = (seen_by(a, s, clamp64(r0 + kRows - 1, 0, s.n - 1)) + KT - 1) / KT;
  const bool all = sizeof(T) == 2 && total <= ST;  // delta from all of the keys
  int from = 0, steps = total;                     // this part's: from .. steps - 1
  if constexpr (SPLIT) {
    from = all ? 0 : (int)((int64_t)total * part / parts);
    steps = all ? (part == 0 ? total : 0) : (int)((int64_t)total * (part + 1) / parts);
  }
  Ld lk, lv;
  lk.init(tid, a.k_rs);
  lv.init(tid, a.v_rs);
  const uint32_t dst = lds0 + wave * 1024;
  u32x4 rk = {}, rv = {};
  uint32_t to = 0;
  auto prepare = [&](int i) {
    const int64_t j = (int64_t)i * KT;
    rk = lk.range(k + j * a.k_rs, s.m - j, a.k_rs, a.dh);
    rv = lv.range(v + j * a.v_rs, s.m - j, a.v_rs, a.dh);
    to = dst + (i & (ST - 1)) * 2 * Ld::kBytes;
  };
  auto piece = [&](int q) {
    if (q < Ld::kRounds) lk.round(q, rk, a.dh, to);
    else lv.round(q - Ld::kRounds, rv, a.dh, to + Ld::kBytes);
  };
  constexpr int kPieces = 2 * Ld::kRounds;
  auto fetch = [&](int i) {
    prepare(i);
#pragma unroll
    for (int q = 0; q < kPieces; ++q) piece(q);
  };
  using Op = Ahead<T, DH>;
  f32x16 acc[Ti::kNDB] = {};
  if (steps > from) {
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(from + i);
  }
  float delta = 0.f;
  if constexpr (sizeof(T) == 2) {
    if (all && steps > 0) {
      fetch(ST - 1);
      wait_and_sync<>();
      for (int i = 0; i * KT < wave_hi; ++i) {
        const uint32_t kt = lds0 + i * 2 * Ld::kBytes;
#pragma unroll
        for (int b = 0; b < NS; ++b) {
          f32x16 x = product<T, DH>(kt + b * 32 * Ti::kRowB, qo, lane);
          const f32x16 g = product<T, DH>(kt + Ld::kBytes + b * 32 * Ti::kRowB, go, lane);
          look(x);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] = exp2_of(__builtin_fmaf(x[e], c, -L)) * g[e];
            delta += i * KT + b * 32 + acc_row(e, lane / 32) < mine ? x[e] : 0.f;
          }
        }
      }
    }
  }
  if (!all) {
    u32x4 oo[Ti::kNT];
    load_own<T, DH>(oo, out + at * a.dh, live, a.dh, lane);
    constexpr int N = 16 / sizeof(T);
    typedef T V __attribute__((ext_vector_type(N)));
#pragma unroll
    for (int i = 0; i < Ti::kNT; ++i) {
      const V x = __builtin_bit_cast(V, go[i]), y = __builtin_bit_cast(V, oo[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) delta += to_f32(x[j]) * to_f32(y[j]);
    }
  }
  delta += other_half(delta);
  for (int i = from; i < steps; ++i) {
    wait_and_sync<(ST - 2) * kPieces>();  // tile i is there, tile i - 1 is done with
    const int j0 = i * KT;
    if (j0 >= wave_hi) {
      fetch(i + ST - 1);
      continue;
    }
    prepare(i + ST - 1);
    const uint32_t kt = lds0 + (i & (ST - 1)) * 2 * Ld::kBytes, vt = kt + Ld::kBytes;
    const bool edge = j0 + KT > wave_lo;
    Op op;
#pragma unroll
    for (int b = 0; b < NS; ++b) {
      const int off = b * 32 * Ti::kRowB;
      const uint32_t kc = Op::cols_at(kt + off, lane), vr = Op::rows_at(vt + off, lane);
      op.rows(Op::rows_at(kt + off, lane));
      pin<T>();
      f32x16 x = op.product(qo, [&](int n) {
        op.row(n, vr);
        spread(b * Op::NT + n, NS * Op::NT, kPieces, piece);
      });
      const f32x16 g = op.product(go, [&](int n) {
        spread(n, Op::NT, Op::S / 2, [&](int e) { op.col(e, kc); });
      });
      look(x);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = exp2_of(__builtin_fmaf(x[e], c, -L)) * (g[e] - delta);
      if (edge) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (j0 + b * 32 + acc_row(e, lane / 32) >= mine) x[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) off_by += x[e];
      const typename Mma<T>::P ds = Mma<T>::pack(x);
      pin<T>();  // x ends here
      op.product_t(acc, ds, [&](int e) {  // (half of its operands are read beside it: registers)
        if (e + Op::S / 2 < Op::S) op.col(e + Op::S / 2, kc);
      });
    }
  }
  wait_and_sync<>();  // no load may reach LDS after the workgroup's end
  off_by += other_half(off_by);
  if (live) {
    const int64_t st = (int64_t)h * a.q_rows + s.q0 + t;
    const float of_row = sizeof(T) == 4 ? ln : (big ? -INFINITY : L0);  // (dk and dv look up what is big)
    if constexpr (SPLIT) {
      const int64_t n = a.q_rows * a.hq;
      store_row<float, Ti::kNDB>(sums + (part * n + at) * a.dh, acc, a.scale, a.dh, lane);
      if (lane < 32) {
        off[part * n + st] = off_by;
        if (part == 0) stat[st] = make_float2(of_row, delta);
      }
    } else {
      store_row<T, Ti::kNDB>(dq + at * a.dh, acc, a.scale, a.dh, lane);
      if (lane < 32) stat[st] = make_float2(of_row, delta + off_by);
    }
  }
}

// The parts' sums in their order, for n elements of dq, four a thread (blockIdx.y == 0), and the delta of n / dh rows.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_dq_join(int parts, int64_t n, int dh, const float* __restrict__ sums,
                                                      const float* __restrict__ off, T* __restrict__ dq,
                                                      float2* __restrict__ stat) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = n / dh;
  if (blockIdx.y == 0) {
    if (i * 4 >= n) return;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < parts; ++p) x += *(const f32x4*)(sums + p * n + i * 4);
    typedef T V4 __attribute__((ext_vector_type(4)));
    V4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = (T)x[j];
    *(V4*)(dq + i * 4) = y;
  } else if (i < rows) {
    float x = 0.f;
    for (int p = 0; p < parts; ++p) x += off[p * rows + i];
    stat[i].y += x;
  }
}


// How the dk/dv kernel lays out a workgroup: 64 keys, two waves for each 32 of them and each of the RS row blocks of
// a stage (32 RS rows of q and dO with their lse and delta; four stages), and P from the first wave of a pair to the
// second, twice.
template <typename T, int DH> struct Dkv {
  static constexpr int kRS = sizeof(T) == 2 && DH > 64 ? 2 : 1;
  static constexpr int kKeys = 64, kQT = 32 * kRS, kStages = 4, kPairs = 2 * kRS, kThreads = kPairs * 128;
  using Ld = Dma<T, DH, kQT, kThreads>;
  static constexpr int kStage = 2 * Ld::kBytes + 512;  // (a multiple of the rows' size)
  static constexpr bool kPack = kRS > 1;  // P as the upper 24 bits of its float32
  static constexpr int kPB = kPack ? 3072 : 4096;
  static constexpr int kP = kStages * kStage, kBytes = kP + kPairs * 2 * kPB;
  static_assert(kBytes <= 160 * 1024 && kPairs * Tile<T, DH>::kNDB * 4096 <= kBytes, "");
};

// P of a wave's tile to LDS and back: 16 values a lane, whole or (PACK) the upper 24 bits of each, four in three words.
template <bool PACK> __device__ inline void put_p(uint32_t at, const f32x16& x) {
  if constexpr (PACK) {
    uint32_t w[12];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a = __float_as_uint(x[4 * e]), b = __float_as_uint(x[4 * e + 1]);
      const uint32_t c = __float_as_uint(x[4 * e + 2]), d = __float_as_uint(x[4 * e + 3]);
      w[3 * e] = __builtin_amdgcn_perm(b, a, 0x05030201);      // a1 a2 a3 b1
      w[3 * e + 1] = __builtin_amdgcn_perm(c, b, 0x06050302);  // b2 b3 c1 c2
      w[3 * e + 2] = __builtin_amdgcn_perm(d, c, 0x07060503);  // c3 d1 d2 d3
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
      *(CUTBCE_LDS u32x4*)(size_t)(at + e * 1024) = u32x4{w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *(CUTBCE_LDS f32x4*)(size_t)(at + e * 1024) = f32x4{x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]};
  }
}
template <bool PACK> __device__ inline float get_p(const u32x4* p, int e) {
  if constexpr (PACK) {
    const int k = e / 4 * 3;
    const uint32_t a = p[k / 4][k % 4], b = p[(k + 1) / 4][(k + 1) % 4], c = p[(k + 2) / 4][(k + 2) % 4];
    switch (e % 4) {
      case 0: return __uint_as_float(a << 8);
      case 1: return __uint_as_float(__builtin_amdgcn_perm(b, a, 0x0504030c));  // 0 a3 b0 b1
      case 2: return __uint_as_float(__builtin_amdgcn_perm(c, b, 0x0403020c));  // 0 b2 b3 c0
      default: return __uint_as_float(c & 0xffffff00u);
    }
  } else {
    return __uint_as_float(p[e / 4][e % 4]);
  }
}

// dk and dv: a workgroup has 64 keys of one sequence and key/value head; the rows of the group's heads stream through
// LDS. One wave would need the sums of dk and dv, k and v of its keys and two score tiles (over 256 registers at
// head_dim 128, one wave per SIMD, and half of them in accumulation registers that vector instructions cannot reach:
// 1.33 ms at 4 x 8192). So a pair of waves shares 32 keys: the first has k and dv (scores, P, P^T dO), the second v
// and dk (dP, dS, dS^T Q) one tile behind, with P handed over in LDS. Two waves per SIMD, one of each kind, hide each
// other's latencies: 640 to 664 us (matrix unit busy 36%; the chain of a turn, scores to P to product, is covered only
// in part by the other wave), 16 us at 128 sequences of up to 200; float32, one sequence of 2,048, 8 heads over 2 of
// 64, in parts: 111 us and 5 for the join. P and dS are rounded to bf16 as operands of the second products, like P in
// the forward: dv off by 0.21 to 0.24% of its norm, dk by 0.23 to 0.24%. Where four stages leave too little room for
// two P's of each pair in float32, its upper 24 bits are handed over: an error of 2^-16, under a hundredth of dS's
// rounding to bf16. (One P, with a second barrier before it is overwritten, was slower; float16 loses what is under
// 2^-38 of a row's sum.)
//
// SPLIT: `parts` workgroups for each key tile and head, with a share of its steps each (dkv_parts).
template <typename T, int DH, bool SPLIT>
__global__ __launch_bounds__((Dkv<T, DH>::kThreads), 2) void k_attn_dkv(Attn a, int parts,
                                                                        const T* __restrict__ dout,
                                                                        const float* __restrict__ lse,
                                                                        const float2* __restrict__ stat,
                                                                        T* __restrict__ dk, T* __restrict__ dv,
                                                                        float* __restrict__ sums) {
  using Ti = Tile<T, DH>;
  using K = Dkv<T, DH>;
  using Ld = typename K::Ld;
  constexpr int QT = K::kQT;
  constexpr bool kLn = sizeof(T) == 4;  // stat has lse itself
  extern __shared__ __align__(1024) char lds[];
  const uint32_t lds0 = uni((uint32_t)(size_t)(CUTBCE_LDS char*)lds);
  const int tid = threadIdx.x, wave = uni(tid / 64), lane = tid % 64, half = lane / 32;
  const int pair = wave % K::kPairs, kw = pair % 2, rw = pair / 2;  // which 32 keys, which rows of a stage
  const bool first = wave < K::kPairs;
  const unsigned part = SPLIT ? blockIdx.x % parts : 0, tile = SPLIT ? blockIdx.x / parts : blockIdx.x;
  const int hk = tile % a.hk;
  const Unit u = find_unit<K::kKeys, false>(a, a.cu_k, a.k_pitch, a.k_rows, tile / a.hk);
  const SeqRange& s = u.s;
  const int64_t j0 = (int64_t)u.tile * K::kKeys;
  if (j0 >= s.cap) return;
  const int64_t j = j0 + kw * 32 + lane % 32;
  const bool key = j < s.m;
  u32x4 own[Ti::kNT];
  load_own<T, DH>(own, first ? (const T*)a.k + s.kb + j * a.k_rs + hk * a.k_hs
                             : (const T*)a.v + s.vb + j * a.v_rs + hk * a.v_hs, key, a.dh, lane);
  const float c = a.scale * kLog2e, ch = a.scale * (0.5f * kLog2e);
  // the first row that sees key x: row t sees it if t >= x - (m - n)
  auto first_row = [&](int64_t x) { return a.causal ? (int)clamp64(x - ((int64_t)s.m - s.n), 0, s.n) : 0; };
  const int mine = first_row(j), wave_hi = first_row(j0 + kw * 32 + 31);
  const int begin = j0 < s.m ? first_row(j0) / QT : 0, end = j0 < s.m ? (s.n + QT - 1) / QT : 0;
  const int total = end > begin ? (end - begin) * a.group : 0;
  const int from = SPLIT ? (int)((int64_t)total * part / parts) : 0;  // the first of this part's steps
  const int steps = SPLIT ? (int)((int64_t)total * (part + 1) / parts) - from : total;
  Ld lq, lg;
  lq.init(tid, a.q_rs);
  lg.init(tid, (int64_t)a.hq * a.dh);
  // The last rows come first, the group's heads in turn for each tile: every key of a sequence sees the last rows, so
  // the workgroups of a sequence read the same tiles at about the same time, through the L2 cache.
  // Workgroups begin with different heads: the rows of one head lie a power of two apart as often as not, and would
  // all come from a few channels of the cache.
  const int turn = (int)(tile / a.hk / 4 % a.group);
  const int h0 = SPLIT ? from % a.group : 0, t0 = end - 1 - (SPLIT ? from / a.group : 0);
  int fh = h0, ft = t0, fi = 0;  // head (from `turn` on), tile and index of the next fetch
  // A fetch in pieces: one load each, to be spread over a turn (together at its beginning they held up the products
  // behind them). Beyond the last tile the range is empty: zeros are loaded.
  constexpr int kPieces = 2 * Ld::kRounds + 1;
  u32x4 rq = {}, rg = {};
  int64_t st_row = 0, st_rem = 0;
  uint32_t st_at = 0;
  auto prepare = [&]() {
    const bool in = fi < steps;
    const int64_t t = (int64_t)ft * QT, rem = in ? s.n - t : 0;
    const int head = in ? hk * a.group + (fh + turn < a.group ? fh + turn : fh + turn - a.group) : 0;
    rq = lq.range((const T*)a.q + (s.q0 + t) * a.q_rs + head * a.q_hs, rem, a.q_rs, a.dh);
    rg = lg.range(dout + ((s.q0 + t) * a.hq + head) * a.dh, rem, (int64_t)a.hq * a.dh, a.dh);
    st_row = (int64_t)head * a.q_rows + s.q0 + t + wave * 32;
    st_rem = rem - wave * 32;
    st_at = lds0 + (uint32_t)(fi % K::kStages) * K::kStage;
    ++fi;
    if (++fh == a.group) fh = 0, --ft;
  };
  auto piece = [&](int k) {
    if (k < Ld::kRounds) lq.round(k, rq, a.dh, st_at + wave * 1024);
    else if (k < 2 * Ld::kRounds) lg.round(k - Ld::kRounds, rg, a.dh, st_at + Ld::kBytes + wave * 1024);
    else if (k == 2 * Ld::kRounds && wave < K::kRS)
      load_pairs(stat + st_row, st_rem, st_at + 2 * Ld::kBytes + wave * 256, lane);
  };
  auto fetch = [&]() {
    prepare();
#pragma unroll
    for (int k = 0; k < kPieces; ++k) piece(k);
  };
  // At turn i the first waves are at tile i and read the rows of tile i + 1 ahead, the second are one tile behind;
  // tile i + 2 is fetched over tile i - 2.
  f32x16 acc[Ti::kNDB] = {};
  const uint32_t px = lds0 + K::kP + pair * 2 * K::kPB + lane * 16;
  const uint32_t rows = lds0 + rw * 32 * Ti::kRowB;
  const uint32_t words = lds0 + 2 * Ld::kBytes + rw * 256 + half * 16;
  auto stage = [](int i) { return (uint32_t)(i % K::kStages) * K::kStage; };
  if (steps > 0) {
    using Op = Ahead<T, DH>;
    Op op;
    // beside the first product: the second one's operands, and the loads of tile i + 2; beside the second: the next
    // rows
    auto beside = [&](int k, uint32_t at) {
      spread(k, Op::NT, Op::S, [&](int e) { op.col(e, at); });
      spread(k, Op::NT, kPieces, piece);
    };
    auto next = [&](int e, uint32_t at) { spread(e, Op::S, Op::NT, [&](int k) { op.row(k, at); }); };
    fetch();
    fetch();
    wait_and_sync<>();
    if (first) {
      op.rows(Op::rows_at(rows, lane));
      int cur = h0, ct = t0;
      for (int i = 0; i < steps; ++i) {
        wait_and_sync<>();
        prepare();
        const uint32_t at = stage(i);
        const int t1 = ct * QT + rw * 32, at_head = cur;
        if (++cur == a.group) cur = 0, --ct;
        f32x4 ld[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) ld[e] = __builtin_bit_cast(f32x4, lds16(words + at + e * 32));
        // one of the 32 rows' words a lane: whether an lse has to be looked up
        const float mark = *(CUTBCE_LDS const float*)(size_t)(words + at - half * 16 + (lane % 32) * 4);
        const uint32_t gc = Op::cols_at(rows + at + Ld::kBytes, lane), nr = Op::rows_at(rows + stage(i + 1), lane);
        bool any_big = false;
        f32x16 x = op.product(own, [&](int k) {
          beside(k, gc);
          if (!kLn && k + 1 == Op::NT) any_big = __any(mark == -INFINITY);
        });
        float f = c;
        if (__builtin_expect(any_big, 0)) {
          const int t = t1 + lane % 32;
          const float l = t < s.n ? lse[(s.q0 + t) * a.hq + hk * a.group + (at_head + turn) % a.group] : 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float L = ld[e / 4][e % 4], big = __shfl(l, acc_row(e, half), 64);
            x[e] = L == -INFINITY ? big_exponent(x[e], ch, big) : __builtin_fmaf(x[e], c, -L);
            ld[e / 4][e % 4] = 0.f;
          }
          f = 1.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          x[e] = exp2_of(kLn ? big_exponent(x[e], ch, ld[e / 4][e % 4]) : __builtin_fmaf(x[e], f, -ld[e / 4][e % 4]));
        if (t1 < wave_hi || t1 + 32 > s.n) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int t = t1 + acc_row(e, half);
            if (t < mine || t >= s.n) x[e] = 0.f;
          }
        }
        put_p<K::kPack>(px + (i & 1) * K::kPB, x);
        op.product_t(acc, Mma<T>::pack(x), [&](int e) { next(e, nr); });
      }
      wait_and_sync<>();
    } else {
      wait_and_sync<>();
      fetch();
      op.rows(Op::rows_at(rows + Ld::kBytes, lane));
      for (int i = 0; i < steps; ++i) {
        wait_and_sync<>();
        prepare();
        const uint32_t at = stage(i);
        f32x4 ld[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) ld[e] = __builtin_bit_cast(f32x4, lds16(words + at + 128 + e * 32));
        u32x4 p[K::kPB / 1024];
#pragma unroll
        for (int e = 0; e < K::kPB / 1024; ++e) p[e] = lds16(px + (i & 1) * K::kPB + e * 1024);
        const uint32_t qc = Op::cols_at(rows + at, lane), nr = Op::rows_at(rows + stage(i + 1) + Ld::kBytes, lane);
        f32x16 g = op.product(own, [&](int k) { beside(k, qc); });
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = get_p<K::kPack>(p, e) * (g[e] - ld[e / 4][e % 4]);
        op.product_t(acc, Mma<T>::pack(g), [&](int e) { next(e, nr); });
      }
    }
    wait_and_sync<>();  // no load may reach LDS after this
  }
  if constexpr (K::kRS > 1) {  // the second rows' sums to the first rows' waves, through LDS
    const uint32_t at = lds0 + ((first ? 0 : 2) + kw) * (Ti::kNDB * 4096) + lane * 16;
#pragma unroll
    for (int d = 0; d < Ti::kNDB; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (rw == 1)
          *(CUTBCE_LDS f32x4*)(size_t)(at + (d * 4 + e) * 1024) =
              f32x4{acc[d][4 * e], acc[d][4 * e + 1], acc[d][4 * e + 2], acc[d][4 * e + 3]};
    wait_and_sync<>();
    if (rw == 1) return;
#pragma unroll
    for (int d = 0; d < Ti::kNDB; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x4 x = __builtin_bit_cast(f32x4, lds16(at + (d * 4 + e) * 1024));
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[d][4 * e + w] += x[w];
      }
  }
  if (j < s.cap) {
    if (!key) {  // a place behind the keys: its own values are not used
#pragma unroll
      for (int d = 0; d < Ti::kNDB; ++d) acc[d] = f32x16{};
    }
    const int64_t row = (s.k0 + j) * a.hk + hk;
    if constexpr (!SPLIT) {
      store_row<T, Ti::kNDB>((first ? dv : dk) + row * a.dh, acc, first ? 1.f : a.scale, a.dh, lane);
    } else {
      store_row<float, Ti::kNDB>(sums + ((2 * part + (first ? 0 : 1)) * a.k_rows * a.hk + row) * a.dh, acc,
                                 first ? 1.f : a.scale, a.dh, lane);
    }
  }
}

// Few key tiles leave CUs idle: the rows (and heads) that a tile meets are then dealt to several workgroups, which
// leave their sums in the workspace for k_attn_dkv_join. At least 256 rows each (fewer are mostly start-up), and no
// more workgroups than two a CU in all. One sequence of 4,096 rows, 8 heads over 1 of 128, bf16: 491 us whole, 111 in 7
// parts with the join; of 2,048, 1 head of 128, float32: 293 and 59; of 600, 2 heads over 1 of 64, bf16: 31 and 18.
int dkv_parts(const Attn& a) {
  const int64_t wgs = (a.k_rows / 64 + a.seqs + 1) * a.hk, most = a.q_pitch * a.group / 256;
  int64_t p = 512 / wgs;
  if (p > most) p = most;
  return (int)(p < 1 ? 1 : p);
}

// The parts' sums in their order: dv (blockIdx.y == 0) and dk of n elements each, four a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_dkv_join(int parts, int64_t n, const float* __restrict__ sums,
                                                       T* __restrict__ dk, T* __restrict__ dv) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) x += *(const f32x4*)(sums + (2 * p + blockIdx.y) * n + i);
  typedef T V4 __attribute__((ext_vector_type(4)));
  V4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = (T)x[j];
  *(V4*)((blockIdx.y ? dk : dv) + i) = y;
}

// ---- few query rows against long key ranges ---------------------------------------------------------------------
// The query heads that share a key/value head, and a sequence's few tokens, are the 32 columns of one tile, so the
// keys are read once for all of them. A workgroup has one part of the keys of one (sequence, key/value head); its
// waves take 32-key blocks in turn, each through an LDS ring of its own (no barriers), and join their results in
// LDS. With more than one part, the parts leave (out, max, sum) in the workspace and k_attn_join joins them in order.
//
// Bound by the cache's bytes: 16 ranges of up to 32,768 keys, 16 heads over 2 of 128, bf16 (403 MB): 80 to 83 us, 4.9
// to 5.0 TB/s, and 4.7 for the join. A workgroup has as many waves as let two of them share a CU's LDS: two of two
// waves took 81 us there, one of four 86. 128 ranges of up to 200 keys, 2 heads of 64: 7.0 us (lengths, first tiles,
// two blocks a wave, the waves' join).
//
// The probabilities go into the second product as two bf16 parts: the kernel waits for memory, and the added matrix
// instructions cost 1 to 3% (80.0 -> 80.7 us and 6.8 -> 7.0 at the sizes above) where one part's rounding was as large
// an error as that of out itself.
//
// bf16 rings have two stages of 32 keys, K and V each. A float32 block keeps the matrix unit busy for about as long as
// its bytes take (32 columns, however few are used), so more waves matter more than more loads in flight: one stage,
// where K of the next block is loaded from the end of the scores on and V from the end of the second product on. 16
// ranges of up to 16,384 keys, 16 heads over 2 of 128 (403 MB): 157 us with two stages and one wave, 105 with one and
// two (3.8 TB/s); 4 heads over 2 of 64: 76 and 53; 100 ranges of up to 200, 2 heads of 128: 37 and 25.

constexpr int kCols = 32;

template <typename T> constexpr int few_stages() { return sizeof(T) == 4 ? 1 : 2; }
template <typename T, int DH> constexpr int few_waves() { return few_stages<T>() * Tile<T, DH>::kRowB > 256 ? 2 : 4; }

// Parts of each key range: enough workgroups for every CU, at least 256 keys in each part (shorter parts are mostly
// start-up: the first tile's latency and the join).
int few_parts(const Attn& a) {
  const int64_t wgs = (int64_t)a.seqs * a.hk;
  int64_t p = cdiv(1024, wgs);
  const int64_t most = cdiv(a.k_pitch, 256);
  if (p > most) p = most;
  return (int)(p < 1 ? 1 : (p > 256 ? 256 : p));
}

template <typename T, int DH>
__global__ __launch_bounds__((few_waves<T, DH>() * 64), 1) void k_attn_few(Attn a, int parts, T* __restrict__ out,
                                                                        float* __restrict__ lse,
                                                                        float* __restrict__ part) {
  using Ti = Tile<T, DH>;
  constexpr int NW = few_waves<T, DH>(), NDB = Ti::kNDB, ST = few_stages<T>();
  using Ld = Dma<T, DH, 32, 64>;
  extern __shared__ __align__(1024) char lds[];
  const int tid = threadIdx.x, wave = uni(tid / 64), lane = tid % 64;
  const uint32_t ring = uni((uint32_t)(size_t)(CUTBCE_LDS char*)lds) + wave * 2 * ST * Ld::kBytes;
  const int pi = blockIdx.x % parts;
  const int64_t bh = blockIdx.x / parts;
  const int hk = (int)(bh % a.hk), seq = (int)(bh / a.hk);
  const SeqRange s0 = seq_range(a, seq);
  SeqRange s = s0;
  s.m = uni(s0.m);
  const int col = lane % 32, cols = s.n * a.group;
  const int t = col / a.group, head = hk * a.group + col % a.group;
  const bool live = col < cols;
  u32x4 qo[Ti::kNT];
  load_own<T, DH>(qo, (const T*)a.q + (s.q0 + t) * a.q_rs + head * a.q_hs, live, a.dh, lane);
  const float ch = half_scale<T, Ti::kNT>(a.scale, qo);
  const int mine = live ? seen_by(a, s, t) : 0, least = seen_by(a, s, 0);
  // this part's 32-key blocks, and the wave's
  const int blocks = (s.m + 31) / 32;
  const int b0 = (int)((int64_t)blocks * pi / parts), b1 = (int)((int64_t)blocks * (pi + 1) / parts);
  const T* k = (const T*)a.k + uni64(s.kb) + hk * a.k_hs;
  const T* v = (const T*)a.v + uni64(s.vb) + hk * a.v_hs;
  Ld lk, lv;
  lk.init(lane, a.k_rs);
  lv.init(lane, a.v_rs);
  auto fetch = [&](const Ld& ld, const T* x, int64_t stride, int b, uint32_t to) {
    const int64_t j = (int64_t)b * 32;
    if constexpr (ST == 2) {
      ld.load(x + j * stride, s.m - j, stride, a.dh, to);
    } else {
      const u32x4 r = ld.range(x + j * stride, s.m - j, stride, a.dh);
#pragma unroll
      for (int q = 0; q < Ld::kRounds; ++q) ld.round(q, r, a.dh, to);
    }
  };
  auto fetch_k = [&](int b, int stage) { fetch(lk, k, a.k_rs, b, ring + stage * 2 * Ld::kBytes); };
  auto fetch_v = [&](int b, int stage) { fetch(lv, v, a.v_rs, b, ring + stage * 2 * Ld::kBytes + Ld::kBytes); };
  // what was read from LDS has arrived, so it may be loaded over
  auto read = []() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
  // all but the last `n` tiles' loads have arrived
  auto arrived = [](auto n) { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(n)::value * Ld::kRounds) : "memory"); };
  using std::integral_constant;
  f32x16 o[NDB] = {};
  Online st;
  int stage = 0;
  if (b0 + wave < b1) {
    fetch_k(b0 + wave, 0);
    fetch_v(b0 + wave, 0);
  }
  for (int b = b0 + wave; b < b1; b += NW, stage ^= ST - 1) {
    const bool more = b + NW < b1;
    if (ST == 2) {
      read();
      if (more) {
        fetch_k(b + NW, stage ^ 1);
        fetch_v(b + NW, stage ^ 1);
        arrived(integral_constant<int, 2>());
      } else {
        arrived(integral_constant<int, 0>());
      }
    } else {
      arrived(integral_constant<int, 1>());
    }
    const uint32_t kt = ring + stage * 2 * Ld::kBytes;
    f32x16 x = product<T, DH>(kt, qo, lane);
    if (ST == 1 && more) {
      read();
      fetch_k(b + NW, 0);
    }
    if (b * 32 + 32 > least) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (b * 32 + acc_row(e, lane / 32) >= mine) x[e] = -INFINITY;
    }
    softmax_step<1, NDB>(&x, ch, st, o);
    if (ST == 1) {
      if (more) arrived(integral_constant<int, 1>());
      else arrived(integral_constant<int, 0>());
    }
    product_t_exact<T, DH>(o, x, kt + Ld::kBytes, lane);
    if (ST == 1 && more) {
      read();
      fetch_v(b + NW, 0);
    }
  }
  st.sum += other_half(st.sum);
  // join the waves: each leaves (max, sum) and its scaled output in LDS, which the rings no longer use
  __syncthreads();
  float* ms = (float*)lds;                  // [NW][2][32]
  float* ot = (float*)(lds + NW * 256);     // [NW][DH][32], one column per row's lane
  if (lane < 32) {
    ms[wave * 64 + lane] = st.half;
    ms[wave * 64 + 32 + lane] = st.sum;
  }
  __syncthreads();
  float mx = -INFINITY, sum = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) mx = fmaxf(mx, ms[w * 64 + col]);
#pragma unroll
  for (int w = 0; w < NW; ++w)
    sum += (ms[w * 64 + col] == -INFINITY ? 0.f : exp2_of(2.f * (ms[w * 64 + col] - mx))) * ms[w * 64 + 32 + col];
  const float f = st.half == -INFINITY ? 0.f : exp2_of(2.f * (st.half - mx));
#pragma unroll
  for (int db = 0; db < NDB; ++db)
#pragma unroll
    for (int e = 0; e < 16; ++e) ot[(wave * DH + db * 32 + acc_row(e, lane / 32)) * 32 + col] = o[db][e] * f;
  __syncthreads();
  // column cc, feature d
  const float inv = mine > 0 ? 1.f / sum : 0.f;
  __shared__ float scale_of[kCols];
  if (wave == 0 && lane < 32) scale_of[lane] = parts == 1 ? inv : 1.f;
  __syncthreads();
  for (int x = tid; x < cols * DH; x += NW * 64) {
    const int cc = x / DH, d = x % DH;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) y += ot[(w * DH + d) * 32 + cc];
    y *= scale_of[cc];
    const int64_t row = s.q0 + cc / a.group;
    const int hd = hk * a.group + cc % a.group;
    if (parts == 1) {
      if (d < a.dh) out[(row * a.hq + hd) * a.dh + d] = (T)y;
    } else {
      part[((bh * parts + pi) * cols + cc) * (DH + 2) + d] = y;
    }
  }
  if (wave == 0 && lane < 32 && live) {
    if (parts > 1) {
      float* p = part + ((bh * parts + pi) * cols + col) * (DH + 2) + DH;
      p[0] = mx;
      p[1] = sum;
    } else if (lse) {
      lse[(s.q0 + t) * a.hq + head] = finish_lse(mx, sum, mine > 0);
    }
  }
}

// One workgroup per (sequence, key/value head, column): the parts' results. Thread i has part i's maximum and sum (at
// most 256 parts), then the threads add the outputs, 32 lanes of four features and eight lots of parts, each in order.
template <typename T, int DH>
__global__ __launch_bounds__(256) void k_attn_join(Attn a, int parts, int cols, T* __restrict__ out,
                                                   float* __restrict__ lse, const float* __restrict__ part) {
  __shared__ float f_of[256], red[4][2], acc[8][DH];
  const int tid = threadIdx.x, wave = tid / 64;
  const int64_t bh = blockIdx.x / cols;
  const int col = (int)(blockIdx.x % cols);
  const SeqRange s = seq_range(a, (int)(bh / a.hk));
  const int t = col / a.group, head = (int)(bh % a.hk) * a.group + col % a.group;
  const bool any = seen_by(a, s, t) > 0;
  const float* p = part + (bh * parts * cols + col) * (DH + 2);
  const int64_t step = (int64_t)cols * (DH + 2);
  const float m = tid < parts ? p[tid * step + DH] : -INFINITY;
  const float l = tid < parts ? p[tid * step + DH + 1] : 0.f;
  float mx = m;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
  if (tid % 64 == 0) red[wave][0] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
  const float f = m == -INFINITY ? 0.f : exp2_of(2.f * (m - mx));
  f_of[tid] = f;
  float sum = f * l;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if (tid % 64 == 0) red[wave][1] = sum;
  __syncthreads();
  sum = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
  const int lot = tid / 32, d = tid % 32 * 4;
  float y[4] = {};
  if (d < DH) {
#pragma unroll 4
    for (int i = lot; i < parts; i += 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] += f_of[i] * p[i * step + d + j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[lot][d + j] = y[j];
  }
  __syncthreads();
  const int64_t at = (s.q0 + t) * a.hq + head;
  if (tid < a.dh) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) z += acc[i][tid];
    out[at * a.dh + tid] = (T)(z * (any ? 1.f / sum : 0.f));
  }
  if (lse && tid == 0) lse[at] = finish_lse(mx, sum, any);
}

// Few query rows: fixed rows per sequence that fill at most one tile's columns with their group's heads.
bool few_rows(const Attn& a) { return !a.cu_q && !a.cu_k && a.q_rows % a.seqs == 0 && a.q_pitch * a.group <= kCols; }

size_t few_bytes(const Attn& a) {
  const int parts = few_parts(a);
  return parts > 1 ? (size_t)a.seqs * a.hk * parts * a.q_pitch * a.group * (128 + 2) * 4 : 0;
}

// Lets kernel F use `bytes` of LDS (the same for every launch of F): set once per device.
template <auto F> hipError_t allow_lds(int bytes) {
  static std::atomic<uint64_t> done{0};
  if (bytes <= 65536) return hipSuccess;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute((const void*)F, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename T, int DH> hipError_t forward_t(const Attn& a, void* out, float* lse, char* ws, hipStream_t st) {
  using Ti = Tile<T, DH>;
  if (few_rows(a)) {
    constexpr int NW = few_waves<T, DH>();
    const int ring = NW * 2 * few_stages<T>() * 32 * Ti::kRowB, join = NW * 256 + NW * DH * 32 * 4;
    const int bytes = ring > join ? ring : join;
    const int parts = few_parts(a), cols = (int)a.q_pitch * a.group;
    const hipError_t e = allow_lds<k_attn_few<T, DH>>(bytes);
    if (e != hipSuccess) return e;
    const int64_t bh = (int64_t)a.seqs * a.hk;
    k_attn_few<T, DH><<<dim3((unsigned)(bh * parts)), dim3(NW * 64), bytes, st>>>(a, parts, (T*)out, lse, (float*)ws);
    if (parts > 1)
      k_attn_join<T, DH><<<dim3((unsigned)(bh * cols)), dim3(256), 0, st>>>(a, parts, cols, (T*)out, lse,
                                                                                   (const float*)ws);
    return hipGetLastError();
  }
  const unsigned units = (unsigned)(units_of(a.q_rows, a.seqs) * a.hq);
  const int bytes = 2 * key_stages<T, DH>() * key_tile<T, DH>() * Ti::kRowB;
  const int parts = row_parts(a);
  if (parts == 1) {
    const hipError_t e = allow_lds<k_attn_fwd<T, DH, false>>(bytes);
    if (e != hipSuccess) return e;
    k_attn_fwd<T, DH, false><<<dim3(units), dim3(256), bytes, st>>>(a, 1, (T*)out, lse, nullptr, nullptr);
  } else {
    const hipError_t e = allow_lds<k_attn_fwd<T, DH, true>>(bytes);
    if (e != hipSuccess) return e;
    const int64_t rows = a.q_rows * a.hq;
    float* sums = (float*)ws;
    float2* stats = (float2*)(sums + parts * rows * a.dh);
    k_attn_fwd<T, DH, true><<<dim3(units * parts), dim3(256), bytes, st>>>(a, parts, (T*)out, lse, sums, stats);
    k_attn_fwd_join<T><<<dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, st>>>(parts, rows, a.dh, sums, stats, (T*)out, lse);
  }
  return hipGetLastError();
}

size_t stat_bytes(const Attn& a) { return cdiv(a.q_rows * a.hq * (int64_t)sizeof(float2), 256) * 256; }

template <typename T, int DH>
hipError_t backward_t(const Attn& a, const void* dout, const void* out, const float* lse, void* dq, void* dk, void* dv,
                      char* ws, hipStream_t st) {
  using Ti = Tile<T, DH>;
  float2* stat = (float2*)ws;
  if (a.q_rows) {
    const unsigned units = (unsigned)(units_of(a.q_rows, a.seqs) * a.hq);
    const int bytes = 2 * key_stages<T, DH>() * key_tile<T, DH>() * Ti::kRowB;
    const int parts = row_parts(a);
    if (parts == 1) {
      const hipError_t e = allow_lds<k_attn_dq<T, DH, false>>(bytes);
      if (e != hipSuccess) return e;
      k_attn_dq<T, DH, false><<<dim3(units), dim3(256), bytes, st>>>(a, 1, (const T*)dout, (const T*)out, lse, (T*)dq,
                                                                    stat, nullptr, nullptr);
    } else {
      const hipError_t e = allow_lds<k_attn_dq<T, DH, true>>(bytes);
      if (e != hipSuccess) return e;
      const int64_t n = a.q_rows * a.hq * a.dh;
      float *sums = (float*)(ws + stat_bytes(a)), *off = sums + parts * n;
      k_attn_dq<T, DH, true><<<dim3(units * parts), dim3(256), bytes, st>>>(a, parts, (const T*)dout, (const T*)out, lse,
                                                                           (T*)dq, stat, sums, off);
      k_attn_dq_join<T><<<dim3((unsigned)cdiv(n, 1024), 2), dim3(256), 0, st>>>(parts, n, a.dh, sums, off, (T*)dq, stat);
    }
  }
  if (a.k_rows) {
    using K = Dkv<T, DH>;
    const int bytes = K::kBytes;
    const unsigned units = (unsigned)(units_of(a.k_rows, a.seqs, K::kKeys) * a.hk);
    const int parts = dkv_parts(a);
    if (parts == 1) {
      const hipError_t e = allow_lds<k_attn_dkv<T, DH, false>>(bytes);
      if (e != hipSuccess) return e;
      k_attn_dkv<T, DH, false><<<dim3(units), dim3(K::kThreads), bytes, st>>>(a, 1, (const T*)dout, lse, stat, (T*)dk,
                                                                             (T*)dv, nullptr);
    } else {
      const hipError_t e = allow_lds<k_attn_dkv<T, DH, true>>(bytes);
      if (e != hipSuccess) return e;
      const int64_t n = a.k_rows * a.hk * a.dh;
      float* sums = (float*)(ws + stat_bytes(a));
      k_attn_dkv<T, DH, true><<<dim3(units * parts), dim3(K::kThreads), bytes, st>>>(a, parts, (const T*)dout, lse, stat,
                                                                                    (T*)dk, (T*)dv, sums);
      k_attn_dkv_join<T><<<dim3((unsigned)cdiv(n, 1024), 2), dim3(256), 0, st>>>(parts, n, sums, (T*)dk, (T*)dv);
    }
  }
  return hipGetLastError();
}

// The kernels are compiled for head_dim rounded up to a multiple of 32.
#define CUTBCE_BY_DIM(F, ...)                                                               \
  (a.dtype == 1 ? (a.dh <= 32   ? F<__bf16, 32>(__VA_ARGS__)                                \
                   : a.dh <= 64 ? F<__bf16, 64>(__VA_ARGS__)                                \
                   : a.dh <= 96 ? F<__bf16, 96>(__VA_ARGS__)                                \
                                : F<__bf16, 128>(__VA_ARGS__))                              \
                : (a.dh <= 32   ? F<float, 32>(__VA_ARGS__)                                 \
                   : a.dh <= 64 ? F<float, 64>(__VA_ARGS__)                                 \
                   : a.dh <= 96 ? F<float, 96>(__VA_ARGS__)                                 \
                                : F<float, 128>(__VA_ARGS__)))

}  // namespace

// A forward launches a workgroup for each tile of rows and head, or (few rows) for each part of a cache and key/value
// head, at most 1,024 more than caches and heads: how many keys there are does not count. The backward is held
// to a tile of 64 rows or keys for each query head, which covers both of its kernels.
bool attention_fits(const Attn& a, bool backward) {
  const int64_t rows = backward && a.k_rows > a.q_rows ? a.k_rows : a.q_rows;
  const int64_t wgs = backward      ? units_of(rows, a.seqs, 64) * a.hq
                      : few_rows(a) ? (int64_t)a.seqs * a.hk
                                    : units_of(rows, a.seqs) * a.hq;
  return wgs < kMaxGrid;
}

// (whether a forward is one of few rows depends on its arrays too: the size covers both)
size_t attention_bytes(const Attn& a, bool backward) {
  const size_t rows = (size_t)a.q_rows * a.hq, keys = (size_t)a.k_rows * a.hk;
  const int parts = row_parts(a), kparts = dkv_parts(a);
  // each part's sums, and two floats a row (the forward) or one (dq)
  const size_t by_rows = parts > 1 ? parts * rows * (a.dh + 2) * sizeof(float) : 0;
  if (backward) {  // dq's are read before those of dk and dv are written
    const size_t by_keys = kparts > 1 ? kparts * 2 * keys * a.dh * sizeof(float) : 0;
    return stat_bytes(a) + (by_rows > by_keys ? by_rows : by_keys);
  }
  const size_t few = a.q_rows % a.seqs == 0 && a.q_pitch * a.group <= kCols ? few_bytes(a) : 0;
  return few > by_rows ? few : by_rows;
}

hipError_t launch_attention_forward(const Attn& a, void* out, float* lse, char* ws, hipStream_t st) {
  return CUTBCE_BY_DIM(forward_t, a, out, lse, ws, st);
}

hipError_t launch_attention_backward(const Attn& a, const void* dout, const void* out, const float* lse, void* dq,
                                     void* dk, void* dv, char* ws, hipStream_t st) {
  return CUTBCE_BY_DIM(backward_t, a, dout, out, lse, dq, dk, dv, ws, st);
}

}  // namespace cutbce
