// Building blocks of the kernels that multiply tiles with 32x32 matrix instructions: tiles of rows in LDS, the direct
// loads that fill them, and the operands that the instructions read from them, row by row or transposed.
#pragma once
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

__host__ __device__ constexpr inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
  static constexpr int kRowB =
      (DH <= 16 && kEsz == 4 ? 16 : DH <= 32 ? 32 : DH <= 64 ? 64 : DH <= 128 ? 128 : 256) * kEsz;
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

// Waits until at most N of the wave's loads are in flight and its LDS accesses are done, then for the workgroup.
template <int N = 0> __device__ inline void wait_and_sync() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The tile's operand of k-step t: the 32 rows from `at`, through the lane's base as above.
template <typename T, int DH> __device__ inline uint32_t base_row(uint32_t at, int lane) {
  using Ti = Tile<T, DH>;
  const int r = lane % 32;
  return at + r * Ti::kRowB + ((lane / 32) ^ Ti::swz(r)) * 16;
}
__device__ inline u32x4 load_row(uint32_t base, int t) { return lds16(base ^ (2 * t * 16)); }

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

}  // namespace

}  // namespace cutbce
