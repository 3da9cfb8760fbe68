// Shared definitions of the sequence encoder's operators (embedding lookup, layer norm, attention): element access,
// the sequences of a packed or cached attention call, and the launchers that encoder_api.hip calls.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace cutbce {

// ---------------------------------------------------------------------------------------------------------
// Elements. bf16 is kept as its 16 bits; f32 -> bf16 rounds to nearest even (v_cvt_pk_bf16_f32).
// ---------------------------------------------------------------------------------------------------------
__device__ inline float to_f32(float x) { return x; }
__device__ inline float to_f32(__bf16 x) { return (float)x; }
template <typename T> __device__ inline T from_f32(float x) { return (T)x; }

// 16 bytes of consecutive elements, aligned to one element only (rows of an odd width).
template <typename T> struct Vec {
  static constexpr int N = 16 / sizeof(T);
  typedef T U __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

template <typename T> __device__ inline void load_vec(const T* p, float* x) {
  const typename Vec<T>::U v = *(const typename Vec<T>::U*)p;
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) x[i] = to_f32(v[i]);
}
template <typename T> __device__ inline void store_vec(T* p, const float* x) {
  typename Vec<T>::U v;
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) v[i] = from_f32<T>(x[i]);
  *(typename Vec<T>::U*)p = v;
}

// The elements at columns c .. c + N - 1 of a row of D (zeros past its end); rows are aligned to one element.
template <typename T> __device__ inline void load_cols(const T* row, int c, int D, float* x) {
  if (c + Vec<T>::N <= D) {
    load_vec(row + c, x);
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) x[i] = c + i < D ? to_f32(row[c + i]) : 0.f;
  }
}
// `past`: the store does not stay in the caches, for outputs that would push out what is still to be read.
template <typename T>
__device__ inline void store_cols(T* row, int c, int D, const float* x, bool past = false) {
  if (c + Vec<T>::N <= D) {
    if (past) {
      typename Vec<T>::U v;
#pragma unroll
      for (int i = 0; i < Vec<T>::N; ++i) v[i] = from_f32<T>(x[i]);
      __builtin_nontemporal_store(v, (typename Vec<T>::U*)(row + c));
    } else {
      store_vec(row + c, x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
      if (c + i < D) row[c + i] = from_f32<T>(x[i]);
  }
}

// Outputs of more than a quarter of the 256 MB memory-side cache go past the caches (measured: a lookup of 262,144 x
// 256 bf16, 134 MB, 44 -> 38 us, layer norm's backward at 65,536 x 2048 195 -> 187 us; at 25,600 x 128, 6.5 MB, no
// difference, and a smaller output is likely still there when the next operator reads it).
inline bool goes_past(int64_t bytes) { return bytes > (int64_t)64 << 20; }

// Workgroups of one launch: a grid has fewer than 2^32 threads in a dimension. What needs more is launched in turns.
constexpr int64_t kMaxGrid = (int64_t)1 << 23;

// ---------------------------------------------------------------------------------------------------------
// Attention: the call's arrays and the ranges of its sequences.
// ---------------------------------------------------------------------------------------------------------
struct Attn {
  const void *q, *k, *v;
  int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs;  // row and head strides in elements
  int64_t k_ss, v_ss;                          // sequence strides where there is no cu_k
  int64_t q_rows, k_rows;
  const int32_t *cu_q, *cu_k, *k_lens;
  int64_t q_pitch, k_pitch;  // rows of each sequence where there is no cu_q / cu_k
  int seqs, hq, hk, group, dh, dtype, causal;
  float scale;
};

// Sequence b (b == seqs: the rows behind the last sequence, without keys): n query rows from q0, m keys from k0, the
// key range's capacity cap >= m; kb and vb are the element offsets of key 0 in k and v. Every range is clamped into
// the arrays.
struct SeqRange {
  int64_t q0, k0, kb, vb;
  int n, m, cap;
};

__device__ inline int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : (x > hi ? hi : x); }

__device__ inline SeqRange seq_range(const Attn& a, int b) {
  SeqRange s;
  int64_t q1, k1;
  const bool tail = b >= a.seqs;
  if (a.cu_q) {
    s.q0 = clamp64(a.cu_q[b], 0, a.q_rows);
    q1 = tail ? a.q_rows : clamp64(a.cu_q[b + 1], s.q0, a.q_rows);
  } else {
    s.q0 = b * a.q_pitch;
    q1 = tail ? a.q_rows : s.q0 + a.q_pitch;
  }
  if (a.cu_k) {
    s.k0 = clamp64(a.cu_k[b], 0, a.k_rows);
    k1 = tail ? a.k_rows : clamp64(a.cu_k[b + 1], s.k0, a.k_rows);
    s.kb = s.k0 * a.k_rs;
    s.vb = s.k0 * a.v_rs;
  } else {
    s.kb = b * a.k_ss;
    s.vb = b * a.v_ss;
    s.k0 = b * a.k_pitch;
    k1 = tail ? a.k_rows : s.k0 + a.k_pitch;
  }
  s.n = (int)(q1 - s.q0);
  s.cap = (int)(k1 - s.k0);
  s.m = tail ? 0 : (a.k_lens ? (int)clamp64(a.k_lens[b], 0, s.cap) : s.cap);
  return s;
}

// ---------------------------------------------------------------------------------------------------------
// Launchers (each returns the hipError_t of its launches).
// ---------------------------------------------------------------------------------------------------------
hipError_t launch_embedding_forward(int64_t n, int64_t V, int D, int dtype, int id_bytes, const void* ids,
                                    const void* table, float scale, void* out, hipStream_t st);
size_t embedding_backward_bytes(int64_t n, int64_t V, int D, int dtype);
hipError_t launch_embedding_backward(int64_t n, int64_t V, int D, int dtype, int id_bytes, const void* ids,
                                     const void* dout, float scale, bool accumulate, void* dtable, char* ws,
                                     hipStream_t st);
hipError_t launch_layer_norm_forward(int64_t rows, int D, int dtype, int pdtype, const void* x, int64_t xs,
                                     const void* w, const void* b, float eps, void* y, float* mean, float* rstd,
                                     hipStream_t st);
size_t layer_norm_backward_bytes(int64_t rows, int D);
hipError_t launch_layer_norm_backward(int64_t rows, int D, int dtype, int pdtype, const void* dy, int64_t dys,
                                      const void* x, int64_t xs, const void* w, const float* mean, const float* rstd,
                                      void* dx, void* dw, void* db, char* ws, hipStream_t st);
bool attention_fits(const Attn& a, bool backward);  // whether one launch of each kernel takes these sizes
size_t attention_bytes(const Attn& a, bool backward);
hipError_t launch_attention_forward(const Attn& a, void* out, float* lse, char* ws, hipStream_t st);
hipError_t launch_attention_backward(const Attn& a, const void* dout, const void* out, const float* lse, void* dq,
                                     void* dk, void* dv, char* ws, hipStream_t st);

}  // namespace cutbce
