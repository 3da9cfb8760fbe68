// The AdamW step over a list of tensors, and the 2-norm of one.
//
//   g' = g min(1, max_norm / (norm + 1e-6)),  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr decay) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// States of 8 bits hold m and r = sqrt(v) (whose range of exponents is half of v's) as e4m3 times a scale for each 256
// elements, their largest magnitude / 448. They are rounded at random: with rounding to nearest a state that changes
// by less than half a step, 3 to 6% of itself, would never move, and v changes by 1 - b2 = 0.1% a step. A positive r is
// never rounded to 0, which would turn its next update into m / eps.
#include "training.h"

namespace cutbce {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Four consecutive elements, aligned to one element; n of them are there.
template <typename T> struct Four {
  typedef T U __attribute__((ext_vector_type(4), aligned(sizeof(T))));
};
template <typename T> __device__ inline void load4(const void* base, int64_t at, int n, float* x) {
  const T* p = (const T*)base + at;
  if (n == 4) {
    const typename Four<T>::U v = *(const typename Four<T>::U*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = to_f32(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
template <typename T> __device__ inline void store4(void* base, int64_t at, int n, const float* x) {
  T* p = (T*)base + at;
  if (n == 4) {
    typename Four<T>::U v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = from_f32<T>(x[i]);
    *(typename Four<T>::U*)p = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_f32<T>(x[i]);
  }
}
__device__ inline void load4(int type, const void* base, int64_t at, int n, float* x) {
  if (type) load4<__bf16>(base, at, n, x);
  else load4<float>(base, at, n, x);
}
__device__ inline void store4(int type, void* base, int64_t at, int n, const float* x) {
  if (type) store4<__bf16>(base, at, n, x);
  else store4<float>(base, at, n, x);
}

// Sixteen consecutive elements, n of them there, the others 0; aligned to one element.
template <typename T> __device__ inline void load16(const void* base, int64_t at, int n, float* x) {
  const T* p = (const T*)base + at;
  constexpr int N = Vec<T>::N;
  if (n == 16) {
#pragma unroll
    for (int i = 0; i < 16; i += N) load_vec(p + i, x + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
template <typename T> __device__ inline void store16(void* base, int64_t at, int n, const float* x) {
  T* p = (T*)base + at;
  constexpr int N = Vec<T>::N;
  if (n == 16) {
#pragma unroll
    for (int i = 0; i < 16; i += N) store_vec(p + i, x + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = from_f32<T>(x[i]);
  }
}
// Sixteen e4m3 bytes.
struct Codes {
  uint32_t w[4];
};
__device__ inline Codes load_codes(const void* base, int64_t at, int n) {
  const uint8_t* p = (const uint8_t*)base + at;
  typedef uint32_t U __attribute__((ext_vector_type(4), aligned(1)));
  Codes c = {};
  if (n == 16) {
    const U v = *(const U*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < n) c.w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  }
  return c;
}
__device__ inline void store_codes(void* base, int64_t at, int n, const Codes& c) {
  uint8_t* p = (uint8_t*)base + at;
  typedef uint32_t U __attribute__((ext_vector_type(4), aligned(1)));
  if (n == 16) {
    *(U*)p = U{c.w[0], c.w[1], c.w[2], c.w[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < n) p[i] = (uint8_t)(c.w[i / 4] >> (8 * (i % 4)));
  }
}
__device__ inline void decode(const Codes& c, float scale, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.w[i], false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.w[i], true);
    x[4 * i] = lo[0] * scale, x[4 * i + 1] = lo[1] * scale, x[4 * i + 2] = hi[0] * scale, x[4 * i + 3] = hi[1] * scale;
  }
}

// 32 bits that look random from a number: the published finalizer of the hash MurmurHash3, two multiplications and
// three shifts, each of which can be undone.
__device__ inline uint32_t hash32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}

// e4m3 of y, |y| <= 448, rounded up in magnitude with the probability random / 2^16 of the part that is cut off; NaN
// stays NaN. `least`: the smallest code of a y that is not 0.
__device__ inline uint32_t encode(float y, uint32_t random, uint32_t least) {
  const uint32_t bits = __float_as_uint(y), a = bits & 0x7fffffffu;
  // (below 2^-6: steps of 2^-9)
  const uint32_t small = (uint32_t)(__uint_as_float(a) * 512.f + (float)random * 0x1p-16f);
  const uint32_t large = ((a + (random << 4)) >> 20) - (120u << 3);
  uint32_t c = a < 0x3c800000u ? small : large;
  c = c > 0x7eu ? 0x7eu : c;
  c = a && c < least ? least : c;
  c = a > 0x7f800000u ? 0x7fu : c;
  return c | ((bits >> 31) << 7);
}

// The largest of 16 lanes' numbers.
__device__ inline uint32_t row_top(uint32_t x) {
#define CUTBCE_TURN(ctrl)                                                                    \
  {                                                                                          \
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, 0xf, 0xf, true); \
    x = y > x ? y : x;                                                                       \
  }
  CUTBCE_TURN(0x128) CUTBCE_TURN(0x124) CUTBCE_TURN(0x122) CUTBCE_TURN(0x121)  // (turned by 8, 4, 2 and 1 lanes)
#undef CUTBCE_TURN
  return x;
}
// A block's values, sixteen a lane, in e4m3 and their scale. NaN counts as the largest (magnitudes are ordered like the
// whole numbers of their bits).
__device__ inline Codes hold(const float* x, const uint32_t* random, int shift, uint32_t least, float* scale) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
    t = a > t ? a : t;
  }
  const float top = __uint_as_float(row_top(t));
  *scale = top * (1.f / 448.f);
  // (what is smaller is held as 0; NaN stays)
  const float f = top > 1e-35f ? 1.f / top * 448.f : (top <= 1e-35f ? 0.f : top);
  Codes c = {};
#pragma unroll
  for (int i = 0; i < 16; ++i) c.w[i / 4] |= encode(x[i] * f, (random[i] >> shift) & 0xffffu, least) << (8 * (i % 4));
  return c;
}

// The states' step, each operation rounded by itself: the random rounding of states of 8 bits turns a difference in the
// last bit into one of a whole step now and then, so this is the same arithmetic that a plain float32 program does.
__device__ inline void advance(const AdamHow& h, float x, bool root, float& m, float& v) {
#pragma clang fp contract(off)
  m = m * h.beta1 + x * h.rest1;
  v = (root ? v * v : v) * h.beta2 + x * x * h.rest2;
}

// What a workgroup needs of the step: its tensor and place in it, and the factors of this step.
struct Place {
  int id;
  int64_t from;
  float clip, keep, rate, c2;
  int32_t t;
};
__device__ inline Place place_of(const AdamArgs& a) {
  Place p;
  const int lane = threadIdx.x % 64;
  const bool here = lane < kListed && a.start[lane < kListed ? lane : 0] <= blockIdx.x;
  p.id = __builtin_amdgcn_readfirstlane(__popcll(__ballot(here)) - 1);
  p.from = (int64_t)(blockIdx.x - a.start[p.id]) * kChunk;
  const AdamHow& h = a.how;
  p.t = *h.step + 1;
  const float c1 = -1.f / expm1f((float)p.t * h.log_beta1);
  p.c2 = sqrtf(-1.f / expm1f((float)p.t * h.log_beta2));
  const float lr = h.lr_at ? *h.lr_at : h.lr;
  p.clip = 1.f;
  if (h.norm) {
    const float x = h.max_norm / (*h.norm + 1e-6f);
    p.clip = x >= 1.f ? 1.f : x;  // (NaN stays)
  }
  p.keep = 1.f - lr * a.e[p.id].decay, p.rate = lr * c1;
  return p;
}

// A workgroup has kChunk elements of one tensor, a lane four consecutive ones at a time. Memory bounds it: 112 million
// bf16 parameters with float32 states, 22 bytes each, take 453 us, 5.45 TB/s.
__global__ __launch_bounds__(256) void k_adamw(AdamArgs a) {
  const Place w = place_of(a);
  const AdamEntry& e = a.e[w.id];
  const AdamHow& h = a.how;
#pragma unroll
  for (int u = 0; u < kChunk / 1024; ++u) {
    const int64_t at = w.from + u * 1024 + threadIdx.x * 4;
    const int64_t left = e.n - at;
    if (left <= 0) break;
    const int n = left >= 4 ? 4 : (int)left;
    float p[4], g[4], m[4], v[4];
    load4(e.g_type, e.g, at, n, g);
    if (e.master) load4<float>(e.master, at, n, p);
    else load4(e.p_type, e.p, at, n, p);
    load4<float>(e.m, at, n, m);
    load4<float>(e.v, at, n, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      advance(h, g[i] * w.clip, false, m[i], v[i]);
      p[i] = p[i] * w.keep - w.rate * m[i] / (sqrtf(v[i]) * w.c2 + h.eps);
    }
    store4<float>(e.m, at, n, m);
    store4<float>(e.v, at, n, v);
    if (e.master) store4<float>(e.master, at, n, p);
    store4(e.p_type, e.p, at, n, p);
  }
}

// The same with states of 8 bits: a lane has sixteen consecutive elements and 16 lanes a block, so that what a block
// costs, the largest of its lanes and two quotients, is shared by many elements.
__global__ __launch_bounds__(256, 4) void k_adamw8(AdamArgs a) {
  const Place w = place_of(a);
  const AdamEntry& e = a.e[w.id];
  const AdamHow& h = a.how;
  const uint32_t key = hash32(hash32(h.seed ^ hash32((uint32_t)w.t)) + a.first + w.id);
  const int64_t at = w.from + threadIdx.x * 16, left = e.n - at, block = at / kBlock8;
  if (block * kBlock8 >= e.n) return;  // (all of the block's lanes)
  const int n = left >= 16 ? 16 : (left > 0 ? (int)left : 0);
  float p[16], g[16], m[16], r[16];
  if (e.g_type) load16<__bf16>(e.g, at, n, g);
  else load16<float>(e.g, at, n, g);
  if (e.master || !e.p_type) load16<float>(e.master ? (const void*)e.master : e.p, at, n, p);
  else load16<__bf16>(e.p, at, n, p);
  decode(load_codes(e.m, at, n), e.ms[block], m);
  decode(load_codes(e.v, at, n), e.vs[block], r);
  uint32_t random[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    advance(h, g[i] * w.clip, true, m[i], r[i]);
    r[i] = sqrtf(r[i]);
    // (the quotient to one unit in its last place: it only moves p)
    p[i] = p[i] * w.keep - w.rate * m[i] * __builtin_amdgcn_rcpf(r[i] * w.c2 + h.eps);
    random[i] = hash32(key + (uint32_t)(at + i));
    if (i >= n) m[i] = r[i] = 0.f;
  }
  float ms, vs;
  const Codes cm = hold(m, random, 0, 0, &ms), cv = hold(r, random, 16, 1, &vs);
  store_codes(e.m, at, n, cm);
  store_codes(e.v, at, n, cv);
  if (threadIdx.x % 16 == 0) e.ms[block] = ms, e.vs[block] = vs;
  if (e.master) store16<float>(e.master, at, n, p);
  if (e.p_type) store16<__bf16>(e.p, at, n, p);
  else store16<float>(e.p, at, n, p);
}

__global__ void k_step(int32_t* step) { *step += 1; }

// Sums of squares in float64: nothing overflows, and a long sum keeps its digits.
__device__ inline double block_sum(double s) {
  __shared__ double part[16];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = s;
  __syncthreads();
  s = 0;
  for (int i = 0; i < (int)blockDim.x / 64; ++i) s += part[i];
  return s;
}

template <typename T> __device__ inline double squares(const void* g, int64_t from, int64_t n) {
  double s = 0;
  constexpr int N = Vec<T>::N;
  const T* p = (const T*)g + from;
  const int64_t left = n - from < kNormChunk ? n - from : kNormChunk;
  int64_t i = threadIdx.x * N;
#pragma unroll 4
  for (; i + N <= left; i += 256 * N) {
    float x[N];
    load_vec(p + i, x);
#pragma unroll
    for (int j = 0; j < N; ++j) s += (double)x[j] * (double)x[j];
  }
  for (; i < left; ++i) {
    const double x = to_f32(p[i]);
    s += x * x;
  }
  return s;
}

__global__ __launch_bounds__(256) void k_norm(NormArgs a) {
  const int lane = threadIdx.x % 64;
  int id = 0;
#pragma unroll
  for (int k = 0; k < kNormListed / 64; ++k) id += __popcll(__ballot(a.start[k * 64 + lane] <= blockIdx.x));
  id = __builtin_amdgcn_readfirstlane(id - 1);
  const int64_t from = (int64_t)(blockIdx.x - a.start[id]) * kNormChunk;
  double s = a.type[id] ? squares<__bf16>(a.g[id], from, a.n[id]) : squares<float>(a.g[id], from, a.n[id]);
  s = block_sum(s);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void k_norm_join(const double* partials, int64_t n, float* norm) {
  double s = 0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += partials[i];
  s = block_sum(s);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, unsigned blocks, bool bits8, hipStream_t st) {
  if (bits8) k_adamw8<<<blocks, 256, 0, st>>>(a);
  else k_adamw<<<blocks, 256, 0, st>>>(a);
  return hipGetLastError();
}
hipError_t launch_step(int32_t* step, hipStream_t st) {
  k_step<<<1, 1, 0, st>>>(step);
  return hipGetLastError();
}
hipError_t launch_norm(const NormArgs& a, unsigned blocks, hipStream_t st) {
  k_norm<<<blocks, 256, 0, st>>>(a);
  return hipGetLastError();
}
hipError_t launch_norm_join(const double* partials, int64_t n, float* norm, hipStream_t st) {
  k_norm_join<<<1, 1024, 0, st>>>(partials, n, norm);
  return hipGetLastError();
}

}  // namespace cutbce
