// Layer norm of rows and its gradients.
//
//   y = (x - mean) * rstd * w + b
//   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)),  g = dy * w,  xhat = (x - mean) * rstd
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy
//
// The weight's gradients are summed in two steps without atomics: each workgroup sums a fixed set of rows into its
// partial [2][D], a second kernel adds the partials of each column in order.
#include "encoder.h"

namespace cutbce {

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kPartRows = 512;  // most workgroups whose partial sums are joined

__device__ inline float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

template <typename P> __device__ inline float param(const P* p, int c, float other) { return p ? to_f32(p[c]) : other; }

// One wave per row.
template <typename T, typename P>
__global__ __launch_bounds__(256) void k_norm(int64_t rows, int D, const T* __restrict__ x, int64_t xs,
                                              const P* __restrict__ w, const P* __restrict__ b, float eps,
                                              T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  const int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int lane = threadIdx.x % 64;
  if (r >= rows) return;
  const T* row = x + r * xs;
  float s = 0.f;
  for (int c = lane; c < D; c += 64) s += to_f32(row[c]);
  const float m = wave_sum(s) / D;
  float q = 0.f;
  for (int c = lane; c < D; c += 64) {
    const float d = to_f32(row[c]) - m;
    q += d * d;
  }
  const float inv = 1.f / sqrtf(wave_sum(q) / D + eps);
  for (int c = lane; c < D; c += 64)
    y[r * D + c] = from_f32<T>((to_f32(row[c]) - m) * inv * param(w, c, 1.f) + param(b, c, 0.f));
  if (mean && lane == 0) {
    mean[r] = m;
    rstd[r] = inv;
  }
}

template <typename T, typename P>
__global__ __launch_bounds__(256) void k_norm_dx(int64_t rows, int D, const T* __restrict__ dy, int64_t dys,
                                                 const T* __restrict__ x, int64_t xs, const P* __restrict__ w,
                                                 const float* __restrict__ mean, const float* __restrict__ rstd,
                                                 T* __restrict__ dx) {
  const int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int lane = threadIdx.x % 64;
  if (r >= rows) return;
  const float m = mean[r], inv = rstd[r];
  float s = 0.f, t = 0.f;
  for (int c = lane; c < D; c += 64) {
    const float g = to_f32(dy[r * dys + c]) * param(w, c, 1.f);
    s += g;
    t += g * ((to_f32(x[r * xs + c]) - m) * inv);
  }
  s = wave_sum(s) / D;
  t = wave_sum(t) / D;
  for (int c = lane; c < D; c += 64) {
    const float g = to_f32(dy[r * dys + c]) * param(w, c, 1.f);
    dx[r * D + c] = from_f32<T>(inv * (g - s - (to_f32(x[r * xs + c]) - m) * inv * t));
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_part(int64_t rows, int D, const T* __restrict__ dy, int64_t dys,
                                                   const T* __restrict__ x, int64_t xs, const float* __restrict__ mean,
                                                   const float* __restrict__ rstd, float* __restrict__ part) {
  const int c = blockIdx.y * 256 + threadIdx.x;
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

template <typename P>
__global__ __launch_bounds__(256) void k_norm_join(int parts, int D, const float* __restrict__ part, P* __restrict__ dw,
                                                   P* __restrict__ db) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  float a = 0.f, b = 0.f;
  for (int k = 0; k < parts; ++k) {
    a += part[((int64_t)k * 2 + 0) * D + c];
    b += part[((int64_t)k * 2 + 1) * D + c];
  }
  if (dw) dw[c] = from_f32<P>(a);
  if (db) db[c] = from_f32<P>(b);
}

int parts_of(int64_t rows) { return (int)(rows < kPartRows ? rows : kPartRows); }

template <typename T, typename P>
hipError_t forward_t(int64_t rows, int D, const void* x, int64_t xs, const void* w, const void* b, float eps, void* y,
                     float* mean, float* rstd, hipStream_t st) {
  k_norm<T, P><<<dim3((unsigned)cdiv(rows, 4)), dim3(256), 0, st>>>(rows, D, (const T*)x, xs, (const P*)w, (const P*)b,
                                                                    eps, (T*)y, mean, rstd);
  return hipGetLastError();
}

template <typename T, typename P>
hipError_t backward_t(int64_t rows, int D, const void* dy, int64_t dys, const void* x, int64_t xs, const void* w,
                      const float* mean, const float* rstd, void* dx, void* dw, void* db, char* ws, hipStream_t st) {
  if (dx && rows > 0)
    k_norm_dx<T, P><<<dim3((unsigned)cdiv(rows, 4)), dim3(256), 0, st>>>(rows, D, (const T*)dy, dys, (const T*)x, xs,
                                                                         (const P*)w, mean, rstd, (T*)dx);
  if (dw || db) {
    const int parts = parts_of(rows);
    if (parts)
      k_norm_part<T><<<dim3(parts, (unsigned)cdiv(D, 256)), dim3(256), 0, st>>>(rows, D, (const T*)dy, dys,
                                                                                (const T*)x, xs, mean, rstd, (float*)ws);
    k_norm_join<P><<<dim3((unsigned)cdiv(D, 256)), dim3(256), 0, st>>>(parts, D, (const float*)ws, (P*)dw, (P*)db);
  }
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

size_t layer_norm_backward_bytes(int64_t rows, int D) { return (size_t)parts_of(rows) * 2 * D * sizeof(float); }

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
