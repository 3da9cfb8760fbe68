// Causal attention over packed sequences or a key/value cache, with grouped heads, and its gradients.
//
//   out = softmax(s q k^T) v, row t of a sequence of n rows and m keys seeing the keys j <= t + m - n
//   P = exp(s q k^T - lse), dP = dO v^T, delta = rowsum(dO * out), dS = P * (dP - delta)
//   dv = P^T dO, dk = s dS^T q, dq = s dS k, dk and dv summed over the query heads that share them
#include "encoder.h"

namespace cutbce {

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ inline float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}
__device__ inline float wave_max(float x) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor(x, o, 64));
  return x;
}

template <typename T> __device__ inline float dot(const T* x, const T* y, int d) {
  float s = 0.f;
  for (int i = 0; i < d; ++i) s += to_f32(x[i]) * to_f32(y[i]);
  return s;
}

// One wave per (row, head): the lanes take 64 keys at a time for the scores and the features for the output.
template <typename T> __global__ __launch_bounds__(256) void k_attn_fwd(Attn a, T* __restrict__ out,
                                                                        float* __restrict__ lse) {
  const int lane = threadIdx.x % 64;
  const int64_t id = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int64_t r = id / a.hq;
  const int h = (int)(id % a.hq), hk = h / a.group, dh = a.dh;
  if (r >= a.q_rows) return;
  const SeqRange s = seq_range(a, seq_of_row(a.cu_q, a.q_pitch, a.seqs, r));
  const int64_t t = r - s.q0;
  int64_t seen = t < 0 || t >= s.n ? 0 : (a.causal ? t + s.m - s.n + 1 : s.m);
  const T* q = (const T*)a.q + r * a.q_rs + h * a.q_hs;
  const T* k = (const T*)a.k + s.kb + hk * a.k_hs;
  const T* v = (const T*)a.v + s.vb + hk * a.v_hs;
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int64_t j0 = 0; j0 < seen; j0 += 64) {
    const bool live = j0 + lane < seen;
    const float z = live ? a.scale * dot(q, k + (j0 + lane) * a.k_rs, dh) : -INFINITY;
    const float mn = fmaxf(m, wave_max(z));
    const float c = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = live && mn != -INFINITY ? expf(z - mn) : 0.f;
    m = mn;
    l = l * c + wave_sum(p);
    o0 *= c;
    o1 *= c;
    const int cnt = (int)(seen - j0 < 64 ? seen - j0 : 64);
    for (int j = 0; j < cnt; ++j) {
      const float pj = __shfl(p, j, 64);
      const T* vj = v + (j0 + j) * a.v_rs;
      if (lane < dh) o0 += pj * to_f32(vj[lane]);
      if (lane + 64 < dh) o1 += pj * to_f32(vj[lane + 64]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (seen > 0 ? l / l : 0.f);
  T* o = out + (r * a.hq + h) * dh;
  if (lane < dh) o[lane] = from_f32<T>(o0 * inv);
  if (lane + 64 < dh) o[lane + 64] = from_f32<T>(o1 * inv);
  if (lse && lane == 0) lse[r * a.hq + h] = seen > 0 ? m + logf(l) : -INFINITY;
}

// delta[row][head] = dO . out
template <typename T>
__global__ __launch_bounds__(256) void k_attn_delta(int64_t n, int dh, const T* __restrict__ dout,
                                                    const T* __restrict__ out, float* __restrict__ delta) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) delta[i] = dot(dout + i * dh, out + i * dh, dh);
}

template <typename T>
__global__ __launch_bounds__(256) void k_attn_dq(Attn a, const T* __restrict__ dout, const float* __restrict__ lse,
                                                 const float* __restrict__ delta, T* __restrict__ dq) {
  const int lane = threadIdx.x % 64;
  const int64_t id = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int64_t r = id / a.hq;
  const int h = (int)(id % a.hq), hk = h / a.group, dh = a.dh;
  if (r >= a.q_rows) return;
  const SeqRange s = seq_range(a, seq_of_row(a.cu_q, a.q_pitch, a.seqs, r));
  const int64_t t = r - s.q0;
  const int64_t seen = t < 0 || t >= s.n ? 0 : (a.causal ? t + s.m - s.n + 1 : s.m);
  const T* q = (const T*)a.q + r * a.q_rs + h * a.q_hs;
  const T* g = dout + (r * a.hq + h) * dh;
  const T* k = (const T*)a.k + s.kb + hk * a.k_hs;
  const T* v = (const T*)a.v + s.vb + hk * a.v_hs;
  const float L = lse[r * a.hq + h], dl = delta[r * a.hq + h];
  float x0 = 0.f, x1 = 0.f;
  for (int64_t j0 = 0; j0 < seen; j0 += 64) {
    const bool live = j0 + lane < seen;
    float ds = 0.f;
    if (live) {
      const float p = expf(a.scale * dot(q, k + (j0 + lane) * a.k_rs, dh) - L);
      ds = p * (dot(g, v + (j0 + lane) * a.v_rs, dh) - dl);
    }
    const int cnt = (int)(seen - j0 < 64 ? seen - j0 : 64);
    for (int j = 0; j < cnt; ++j) {
      const float d = __shfl(ds, j, 64);
      const T* kj = k + (j0 + j) * a.k_rs;
      if (lane < dh) x0 += d * to_f32(kj[lane]);
      if (lane + 64 < dh) x1 += d * to_f32(kj[lane + 64]);
    }
  }
  T* o = dq + (r * a.hq + h) * dh;
  if (lane < dh) o[lane] = from_f32<T>(x0 * a.scale);
  if (lane + 64 < dh) o[lane + 64] = from_f32<T>(x1 * a.scale);
}

// One wave per (key, key/value head): the lanes take 64 rows at a time, the group's heads in turn.
template <typename T>
__global__ __launch_bounds__(256) void k_attn_dkv(Attn a, const T* __restrict__ dout, const float* __restrict__ lse,
                                                  const float* __restrict__ delta, T* __restrict__ dk,
                                                  T* __restrict__ dv) {
  const int lane = threadIdx.x % 64;
  const int64_t id = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int64_t r = id / a.hk;
  const int hk = (int)(id % a.hk), dh = a.dh;
  if (r >= a.k_rows) return;
  const SeqRange s = seq_range(a, seq_of_row(a.cu_k, a.k_pitch, a.seqs, r));
  const int64_t j = r - s.k0;
  const bool key = j >= 0 && j < s.m;
  int64_t t0 = a.causal ? j - (s.m - s.n) : 0;  // the first row that sees the key
  if (t0 < 0) t0 = 0;
  const T* k = (const T*)a.k + s.kb + j * a.k_rs + hk * a.k_hs;
  const T* v = (const T*)a.v + s.vb + j * a.v_rs + hk * a.v_hs;
  float k0 = 0.f, k1 = 0.f, v0 = 0.f, v1 = 0.f;
  if (key)
    for (int h = hk * a.group; h < (hk + 1) * a.group; ++h) {
      const T* q = (const T*)a.q + s.q0 * a.q_rs + h * a.q_hs;
      for (int64_t i0 = t0; i0 < s.n; i0 += 64) {
        float p = 0.f, ds = 0.f;
        if (i0 + lane < s.n) {
          const int64_t at = (s.q0 + i0 + lane) * a.hq + h;
          p = expf(a.scale * dot(q + (i0 + lane) * a.q_rs, k, dh) - lse[at]);
          ds = p * (dot(dout + at * dh, v, dh) - delta[at]);
        }
        const int cnt = (int)(s.n - i0 < 64 ? s.n - i0 : 64);
        for (int i = 0; i < cnt; ++i) {
          const float pi = __shfl(p, i, 64), di = __shfl(ds, i, 64);
          const T* qi = q + (i0 + i) * a.q_rs;
          const T* gi = dout + ((s.q0 + i0 + i) * a.hq + h) * dh;
          if (lane < dh) k0 += di * to_f32(qi[lane]), v0 += pi * to_f32(gi[lane]);
          if (lane + 64 < dh) k1 += di * to_f32(qi[lane + 64]), v1 += pi * to_f32(gi[lane + 64]);
        }
      }
    }
  const int64_t o = (r * a.hk + hk) * dh;
  if (lane < dh) dk[o + lane] = from_f32<T>(k0 * a.scale), dv[o + lane] = from_f32<T>(v0);
  if (lane + 64 < dh) dk[o + lane + 64] = from_f32<T>(k1 * a.scale), dv[o + lane + 64] = from_f32<T>(v1);
}

template <typename T> hipError_t forward_t(const Attn& a, void* out, float* lse, hipStream_t st) {
  k_attn_fwd<T><<<dim3((unsigned)cdiv(a.q_rows * a.hq, 4)), dim3(256), 0, st>>>(a, (T*)out, lse);
  return hipGetLastError();
}

template <typename T>
hipError_t backward_t(const Attn& a, const void* dout, const void* out, const float* lse, void* dq, void* dk, void* dv,
                      char* ws, hipStream_t st) {
  float* delta = (float*)ws;
  const int64_t n = a.q_rows * a.hq;
  if (n) {
    k_attn_delta<T><<<dim3((unsigned)cdiv(n, 256)), dim3(256), 0, st>>>(n, a.dh, (const T*)dout, (const T*)out, delta);
    k_attn_dq<T><<<dim3((unsigned)cdiv(n, 4)), dim3(256), 0, st>>>(a, (const T*)dout, lse, delta, (T*)dq);
  }
  if (a.k_rows)
    k_attn_dkv<T><<<dim3((unsigned)cdiv(a.k_rows * a.hk, 4)), dim3(256), 0, st>>>(a, (const T*)dout, lse, delta,
                                                                                  (T*)dk, (T*)dv);
  return hipGetLastError();
}

}  // namespace

size_t attention_bytes(const Attn& a, bool backward) { return backward ? (size_t)a.q_rows * a.hq * 4 : 0; }

hipError_t launch_attention_forward(const Attn& a, void* out, float* lse, char*, hipStream_t st) {
  return a.dtype == 1 ? forward_t<__bf16>(a, out, lse, st) : forward_t<float>(a, out, lse, st);
}

hipError_t launch_attention_backward(const Attn& a, const void* dout, const void* out, const float* lse, void* dq,
                                     void* dk, void* dv, char* ws, hipStream_t st) {
  return a.dtype == 1 ? backward_t<__bf16>(a, dout, out, lse, dq, dk, dv, ws, st)
                      : backward_t<float>(a, dout, out, lse, dq, dk, dv, ws, st);
}

}  // namespace cutbce
