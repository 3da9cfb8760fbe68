// Layer norm of rows and its gradients.
//
//   y = (x - mean) * rstd * w + b
//   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)),  g = dy * w,  xhat = (x - mean) * rstd
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy
//
// Both directions are bound by memory, so a row is read once: a group of G lanes (a power of two, or the whole
// workgroup) holds it in registers, C 16-byte chunks a lane, and the sums go through lane exchanges (LDS between
// waves). The variance is the mean square of x - mean, from the registers, so a mean far from zero costs nothing.
// The backward adds its rows' share of dw and db in registers on the same pass; each workgroup takes a fixed range of
// rows and leaves one partial [2][D], and a second kernel adds the partials of each column in a fixed order: no
// atomics, the same bits every time.
//
// Rows wider than kWide columns are read several times by a workgroup each, from the caches.
#include "encoder.h"

namespace cutbce {

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kWide = 8192;      // widest row that a workgroup holds: 256 lanes of 32 elements
constexpr int kMaxParts = 1536;  // most partials of the weight's gradients
constexpr int kJoinCols = 16;

template <typename P> __device__ inline float param(const P* p, int c, float other) { return p ? to_f32(p[c]) : other; }
// columns c .. of the weight (or bias), `other` without one
template <typename P, int N> __device__ inline void params(const P* p, int c, int D, float other, float* x) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = other;
  } else if (c + N <= D) {
    constexpr int M = Vec<P>::N < N ? Vec<P>::N : N;
    typedef P V __attribute__((ext_vector_type(M), aligned(sizeof(P))));
#pragma unroll
    for (int k = 0; k < N; k += M) {
      const V v = *(const V*)(p + c + k);
#pragma unroll
      for (int i = 0; i < M; ++i) x[k + i] = to_f32(v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = c + i < D ? to_f32(p[c + i]) : 0.f;
  }
}

// Sums over a group of G lanes; all of them get the result. G == kThreads: over the workgroup.
__device__ inline void group_sum(float& a, float& b, int G, float (*sh)[2]) {
  for (int o = (G < 64 ? G : 64) / 2; o >= 1; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if (G == kThreads) {
    const int wave = threadIdx.x / 64;
    __syncthreads();  // the previous sum has been read
    if (threadIdx.x % 64 == 0) sh[wave][0] = a, sh[wave][1] = b;
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) a += sh[w][0], b += sh[w][1];
  }
}

// Forward. C chunks of N elements a lane: chunk k of lane s covers the columns (k * G + s) * N .. + N - 1. 65,536 x
// 2048 bf16 (64 lanes of 32): 122 us, 4.4 TB/s read and written (a large copy 4.9); lanes of 16 elements, two waves a
// row, 157. 25,600 x 128: 7.1 us, 1.8 TB/s, start-up and two rounds of exchanges. 32 x 64: 2.4 us (an empty kernel
// 1.4).
template <typename T, typename P, int C>
__global__ __launch_bounds__(kThreads) void k_norm(int64_t rows, int D, int G, const T* __restrict__ x, int64_t xs,
                                                   const P* __restrict__ w, const P* __restrict__ b, float eps,
                                                   T* __restrict__ y, float* __restrict__ mean,
                                                   float* __restrict__ rstd) {
  constexpr int N = Vec<T>::N;
  __shared__ float sh[kWaves][2];
  const int s = threadIdx.x % G;
  const int64_t r = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
  if (r >= rows) return;  // whole groups only (a group of kThreads is the workgroup)
  float v[C][N];
  float sum = 0.f, q = 0.f;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    load_cols(x + r * xs, (k * G + s) * N, D, v[k]);
#pragma unroll
    for (int i = 0; i < N; ++i) sum += v[k][i];
  }
  float none = 0.f;
  group_sum(sum, none, G, sh);
  const float m = sum / D;
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = v[k][i] - m;
      q += (k * G + s) * N + i < D ? d * d : 0.f;
    }
  group_sum(q, none, G, sh);
  const float inv = 1.f / sqrtf(q / D + eps);
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const int c = (k * G + s) * N;
    if (c < D) {
      float pw[N], pb[N];
      params<P, N>(w, c, D, 1.f, pw);
      params<P, N>(b, c, D, 0.f, pb);
#pragma unroll
      for (int i = 0; i < N; ++i) v[k][i] = (v[k][i] - m) * inv * pw[i] + pb[i];
      store_cols(y + r * D, c, D, v[k]);
    }
  }
  if (mean && s == 0) {
    mean[r] = m;
    rstd[r] = inv;
  }
}

// One pass over a workgroup's rows: dx, and its share of dw and db. PARAMS: part is wanted. 65,536 x 2048 bf16: 177 us,
// 4.6 TB/s; 25,600 x 128: 11.6 us and 4,097 x 1000 float32: 18.3 us (2.7 TB/s), where a group's two rows come one
// after another, a latency each, with the sums over the groups behind them (workgroups of fewer rows leave more
// partials to join: k_norm_join reads 2 D floats of each, 10 us at 1,536 x 2 x 2048, 4 us at the smaller sizes).
// Loading a row ahead of its turn: 18.9 us and, for the registers, 258 instead of 174 at 65,536 x 2048.
template <typename T, typename P, int C, bool PARAMS>
__global__ __launch_bounds__(kThreads) void k_norm_grad(int64_t rows, int D, int G, const T* __restrict__ dy,
                                                        int64_t dys, const T* __restrict__ x, int64_t xs,
                                                        const P* __restrict__ w, const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, T* __restrict__ dx,
                                                        float* __restrict__ part, bool past) {
  constexpr int N = Vec<T>::N;
  extern __shared__ float acc[];  // [2][D] where PARAMS and a wave holds a row
  __shared__ float sh[kWaves][2];
  const int s = threadIdx.x % G, groups = kThreads / G;
  const int64_t r0 = rows * blockIdx.x / gridDim.x, r1 = rows * (blockIdx.x + 1) / gridDim.x;
  float aw[C][N] = {}, ab[C][N] = {};
  float pw[C][N];
#pragma unroll
  for (int k = 0; k < C; ++k) params<P, N>(w, (k * G + s) * N, D, 1.f, pw[k]);
  for (int64_t r = r0 + threadIdx.x / G; r < r1; r += groups) {
    const float m = mean[r], inv = rstd[r];
    float g[C][N], h[C][N];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      load_cols(dy + r * dys, (k * G + s) * N, D, g[k]);
      load_cols(x + r * xs, (k * G + s) * N, D, h[k]);
    }
    float a = 0.f, t = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        h[k][i] = (h[k][i] - m) * inv;  // past the row's end g is 0
        if (PARAMS) {
          ab[k][i] += g[k][i];
          aw[k][i] += g[k][i] * h[k][i];
        }
        g[k][i] *= pw[k][i];
        a += g[k][i];
        t += g[k][i] * h[k][i];
      }
    if (dx) {
      group_sum(a, t, G, sh);
      a /= D;
      t /= D;
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int i = 0; i < N; ++i) g[k][i] = inv * (g[k][i] - a - h[k][i] * t);
        if ((k * G + s) * N < D) store_cols(dx + r * D, (k * G + s) * N, D, g[k], past);
      }
    }
  }
  if (!PARAMS) return;
  // the lanes that share columns: within a wave by exchanges, between waves one after another in LDS
  for (int o = G; o < 64; o *= 2)
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        aw[k][i] += __shfl_xor(aw[k][i], o, 64);
        ab[k][i] += __shfl_xor(ab[k][i], o, 64);
      }
  float* p = part + (int64_t)blockIdx.x * 2 * D;
  if (G == kThreads) {
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (k * G + s) * N + i;
        if (c < D) p[c] = aw[k][i], p[D + c] = ab[k][i];
      }
    return;
  }
  for (int q = 0; q < kWaves; ++q) {
    if (q == (int)threadIdx.x / 64 && (int)threadIdx.x % 64 < G) {
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = (k * G + s) * N + i;
          if (c < D) {
            acc[c] = (q ? acc[c] : 0.f) + aw[k][i];
            acc[D + c] = (q ? acc[D + c] : 0.f) + ab[k][i];
          }
        }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) p[c] = acc[c];
}

// Rows of any width, a workgroup each, read three times, the second and third from the caches (a row of 8,193 float32
// is 33 KB, and a workgroup reads its own row only), an element a lane at a time: the loads' number bounds it. 4,096 x
// 16,384 bf16: 193 us, 1.4 TB/s of the rows read and written once; float32 213, 2.5. The backward in three launches
// (dx, partials, their join): 220, 122 and 43 us; float32 265, 147 and 46.
template <typename T, typename P>
__global__ __launch_bounds__(kThreads) void k_norm_wide(int D, const T* __restrict__ x, int64_t xs,
                                                        const P* __restrict__ w, const P* __restrict__ b, float eps,
                                                        T* __restrict__ y, float* __restrict__ mean,
                                                        float* __restrict__ rstd) {
  __shared__ float sh[kWaves][2];
  const int64_t r = blockIdx.x;
  const T* row = x + r * xs;
  float sum = 0.f, q = 0.f, none = 0.f;
  for (int c = threadIdx.x; c < D; c += kThreads) sum += to_f32(row[c]);
  group_sum(sum, none, kThreads, sh);
  const float m = sum / D;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const float d = to_f32(row[c]) - m;
    q += d * d;
  }
  group_sum(q, none, kThreads, sh);
  const float inv = 1.f / sqrtf(q / D + eps);
  for (int c = threadIdx.x; c < D; c += kThreads)
    y[r * D + c] = from_f32<T>((to_f32(row[c]) - m) * inv * param(w, c, 1.f) + param(b, c, 0.f));
  if (mean && threadIdx.x == 0) {
    mean[r] = m;
    rstd[r] = inv;
  }
}

template <typename T, typename P>
__global__ __launch_bounds__(kThreads) void k_norm_wide_dx(int D, const T* __restrict__ dy, int64_t dys,
                                                           const T* __restrict__ x, int64_t xs,
                                                           const P* __restrict__ w, const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, T* __restrict__ dx) {
  __shared__ float sh[kWaves][2];
  const int64_t r = blockIdx.x;
  const float m = mean[r], inv = rstd[r];
  float a = 0.f, t = 0.f;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const float g = to_f32(dy[r * dys + c]) * param(w, c, 1.f);
    a += g;
    t += g * ((to_f32(x[r * xs + c]) - m) * inv);
  }
  group_sum(a, t, kThreads, sh);
  a /= D;
  t /= D;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const float g = to_f32(dy[r * dys + c]) * param(w, c, 1.f);
    dx[r * D + c] = from_f32<T>(inv * (g - a - (to_f32(x[r * xs + c]) - m) * inv * t));
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_wide_part(int64_t rows, int D, const T* __restrict__ dy, int64_t dys,
                                                             const T* __restrict__ x, int64_t xs,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd,
                                                             float* __restrict__ part) {
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= D) return;
  const int64_t r0 = rows * blockIdx.x / gridDim.x, r1 = rows * (blockIdx.x + 1) / gridDim.x;
  float dw = 0.f, db = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = to_f32(dy[r * dys + c]);
    db += g;
    dw += g * ((to_f32(x[r * xs + c]) - mean[r]) * rstd[r]);
  }
  part[((int64_t)blockIdx.x * 2 + 0) * D + c] = dw;
  part[((int64_t)blockIdx.x * 2 + 1) * D + c] = db;
}

// dw (columns [0, D)) and db (columns [D, 2D)) from the partials: 16 columns a workgroup, 64 threads a column that
// each add every 64th partial, then the 64 sums in order of a tree.
template <typename P>
__global__ __launch_bounds__(1024) void k_norm_join(int parts, int D, const float* __restrict__ part,
                                                    P* __restrict__ dw, P* __restrict__ db) {
  __shared__ float sh[64][kJoinCols];
  const int col = threadIdx.x % kJoinCols, lane = threadIdx.x / kJoinCols;
  const int64_t c = (int64_t)blockIdx.x * kJoinCols + col;
  float a = 0.f;
  if (c < 2 * (int64_t)D) {
#pragma unroll 8
    for (int k = lane; k < parts; k += 64) a += part[(int64_t)k * 2 * D + c];
  }
  sh[lane][col] = a;
  __syncthreads();
  for (int o = 32; o >= 1; o >>= 1) {
    if (lane < o) sh[lane][col] += sh[lane + o][col];
    __syncthreads();
  }
  if (lane == 0 && c < 2 * (int64_t)D) {
    P* to = c < D ? dw : db;
    if (to) to[c < D ? c : c - D] = from_f32<P>(sh[0][col]);
  }
}

// How a row is held: G lanes of C chunks, the fewest lanes of a wave that give each one chunk, else the wave's 64 with
// up to `most` elements each, else the workgroup's 256. most = 32 in the forward. In the backward, where each element
// brings two sums along, 16: at 65,536 x 2048 bf16 64 lanes of 32 elements took 260 us (251 registers, two waves per
// SIMD), 256 lanes of 8 191 us.
struct Hold {
  int G, C;
};
template <typename T> Hold hold_of(int D, int most) {
  constexpr int N = Vec<T>::N;
  const int chunks = (int)cdiv(D, N);
  Hold h;
  h.G = 1;
  while (h.G < 64 && h.G < chunks) h.G *= 2;
  if (cdiv(chunks, h.G) * N > most) h.G = kThreads;
  h.C = 1;
  while (h.C * h.G < chunks) h.C *= 2;
  return h;
}

// Workgroups of the backward, each with a partial, so that the partials are a small part of what is moved: 32 rows
// each up to 512 columns (8 a group at 512, bf16 2 a group at 128; of 16 columns three groups in four have none), 8
// beyond (2 a group up to 1,024 columns, then all 8), 4 of rows wider than kWide.
int parts_of(int64_t rows, int D) {
  const int per = D > kWide ? 4 : (D > 512 ? 8 : 32);
  const int64_t p = cdiv(rows, per);
  return (int)(p < kMaxParts ? p : kMaxParts);
}

template <typename T, typename P>
hipError_t forward_t(int64_t rows, int D, const void* x, int64_t xs, const void* w, const void* b, float eps, void* y,
                     float* mean, float* rstd, hipStream_t st) {
  if (D > kWide) {
    k_norm_wide<T, P><<<dim3((unsigned)rows), dim3(kThreads), 0, st>>>(D, (const T*)x, xs, (const P*)w, (const P*)b,
                                                                       eps, (T*)y, mean, rstd);
    return hipGetLastError();
  }
  const Hold h = hold_of<T>(D, 32);
  const int per = kThreads / h.G;
  for (int64_t r = 0; r < rows; r += kMaxGrid * per) {
    const int64_t n = rows - r < kMaxGrid * per ? rows - r : kMaxGrid * per;
    const dim3 grid((unsigned)cdiv(n, per));
    float *mr = mean ? mean + r : nullptr, *rr = mean ? rstd + r : nullptr;
#define CUTBCE_NORM(C)                                                                                             \
  k_norm<T, P, C><<<grid, dim3(kThreads), 0, st>>>(n, D, h.G, (const T*)x + r * xs, xs, (const P*)w, (const P*)b, \
                                                   eps, (T*)y + r * D, mr, rr)
    switch (h.C) {
      case 1: CUTBCE_NORM(1); break;
      case 2: CUTBCE_NORM(2); break;
      case 4: CUTBCE_NORM(4); break;
      default:
        if constexpr (sizeof(T) == 4) CUTBCE_NORM(8);
    }
  }
#undef CUTBCE_NORM
  return hipGetLastError();
}

template <typename T, typename P>
hipError_t backward_t(int64_t rows, int D, const void* dy, int64_t dys, const void* x, int64_t xs, const void* w,
                      const float* mean, const float* rstd, void* dx, void* dw, void* db, char* ws, hipStream_t st) {
  const bool params = dw || db;
  int parts = parts_of(rows, D);
  if (parts && D > kWide) {
    if (dx)
      k_norm_wide_dx<T, P><<<dim3((unsigned)rows), dim3(kThreads), 0, st>>>(D, (const T*)dy, dys, (const T*)x, xs,
                                                                            (const P*)w, mean, rstd, (T*)dx);
    if (params)
      k_norm_wide_part<T><<<dim3(parts, (unsigned)cdiv(D, kThreads)), dim3(kThreads), 0, st>>>(
          rows, D, (const T*)dy, dys, (const T*)x, xs, mean, rstd, (float*)ws);
  } else if (parts) {
    const Hold h = hold_of<T>(D, 16);
    // no more workgroups than are resident at once (by the registers that the sums take): at 65,536 x 2048 bf16, 8
    // elements a lane, 1,024 took 195 us, 1,536 177, 2,048 211
    const int epl = h.C * Vec<T>::N, resident = epl <= 8 ? kMaxParts : (epl <= 16 ? 768 : 512);
    if (parts > resident) parts = resident;
    const bool past = goes_past(rows * D * (int64_t)sizeof(T));
    const int lds = params && h.G <= 64 ? 2 * D * (int)sizeof(float) : 0;  // at most 8 KB
#define CUTBCE_GRAD(C)                                                                                               \
  (params ? k_norm_grad<T, P, C, true><<<dim3(parts), dim3(kThreads), lds, st>>>(                                    \
                rows, D, h.G, (const T*)dy, dys, (const T*)x, xs, (const P*)w, mean, rstd, (T*)dx, (float*)ws, past) \
          : k_norm_grad<T, P, C, false><<<dim3(parts), dim3(kThreads), lds, st>>>(                                   \
                rows, D, h.G, (const T*)dy, dys, (const T*)x, xs, (const P*)w, mean, rstd, (T*)dx, (float*)ws, past))
    switch (h.C) {
      case 1: CUTBCE_GRAD(1); break;
      case 2: CUTBCE_GRAD(2); break;
      case 4: CUTBCE_GRAD(4); break;
      default:
        if constexpr (sizeof(T) == 4) CUTBCE_GRAD(8);
    }
#undef CUTBCE_GRAD
  }
  if (params)
    k_norm_join<P><<<dim3((unsigned)cdiv(2 * (int64_t)D, kJoinCols)), dim3(1024), 0, st>>>(
        parts, D, (const float*)ws, (P*)dw, (P*)db);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm_forward(int64_t rows, int D, int dtype, int pdtype, const void* x, int64_t xs,
                                     const void* w, const void* b, float eps, void* y, float* mean, float* rstd,
                                     hipStream_t st) {
  if (dtype == 1)
    return pdtype == 1 ? forward_t<__bf16, __bf16>(rows, D, x, xs, w, b, eps, y, mean, rstd, st)
                       : forward_t<__bf16, float>(rows, D, x, xs, w, b, eps, y, mean, rstd, st);
  return pdtype == 1 ? forward_t<float, __bf16>(rows, D, x, xs, w, b, eps, y, mean, rstd, st)
                     : forward_t<float, float>(rows, D, x, xs, w, b, eps, y, mean, rstd, st);
}

size_t layer_norm_backward_bytes(int64_t rows, int D) { return (size_t)parts_of(rows, D) * 2 * D * sizeof(float); }

hipError_t launch_layer_norm_backward(int64_t rows, int D, int dtype, int pdtype, const void* dy, int64_t dys,
                                      const void* x, int64_t xs, const void* w, const float* mean, const float* rstd,
                                      void* dx, void* dw, void* db, char* ws, hipStream_t st) {
  if (dtype == 1)
    return pdtype == 1 ? backward_t<__bf16, __bf16>(rows, D, dy, dys, x, xs, w, mean, rstd, dx, dw, db, ws, st)
                       : backward_t<__bf16, float>(rows, D, dy, dys, x, xs, w, mean, rstd, dx, dw, db, ws, st);
  return pdtype == 1 ? backward_t<float, __bf16>(rows, D, dy, dys, x, xs, w, mean, rstd, dx, dw, db, ws, st)
                     : backward_t<float, float>(rows, D, dy, dys, x, xs, w, mean, rstd, dx, dw, db, ws, st);
}

}  // namespace cutbce
