// C ABI of the sequence encoder's operators (declared in include/cutbce.h): argument checks and launches.
#include "../../include/cutbce.h"
#include "encoder.h"

using namespace cutbce;

namespace {

constexpr int64_t kMaxRows = 0x7fffffff;
constexpr int64_t kMaxKeys = kMaxRows - 1023;  // keys are counted in 32 bits, up to some tiles past the last
constexpr int64_t kMaxVocab = (int64_t)0x7fffffff - 1024;
constexpr int kMaxDim = 65536;
constexpr int64_t kMaxSorted = (int64_t)1 << 28;  // a workgroup for 32 sorted positions or more, in one launch

bool bad_align(const void* p, size_t a) { return p && ((uintptr_t)p % a) != 0; }
bool known(int dtype) { return dtype == CUTBCE_F32 || dtype == CUTBCE_BF16; }
size_t size_of(int dtype) { return dtype == CUTBCE_BF16 ? 2 : 4; }
cutbce_status of_hip(hipError_t e) { return e == hipSuccess ? CUTBCE_OK : CUTBCE_ERR_HIP; }

cutbce_status check_embedding(int64_t n, int64_t vocab, int dim, int dtype) {
  if (!known(dtype)) return CUTBCE_ERR_DTYPE;
  if (n < 0 || n > kMaxRows || vocab < 1 || vocab > kMaxVocab || dim < 1 || dim > kMaxDim) return CUTBCE_ERR_SHAPE;
  return CUTBCE_OK;
}

cutbce_status check_norm(int64_t rows, int dim, int dtype, int pdtype) {
  if (!known(dtype) || !known(pdtype)) return CUTBCE_ERR_DTYPE;
  if (rows < 0 || rows > kMaxRows || dim < 1 || dim > kMaxDim) return CUTBCE_ERR_SHAPE;
  return CUTBCE_OK;
}

// The call's description as the kernels take it; pointers are not looked at.
cutbce_status make_attn(const cutbce_attention* p, const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_lens,
                        Attn* a) {
  if (!p) return CUTBCE_ERR_NULL;
  if (!known(p->dtype)) return CUTBCE_ERR_DTYPE;
  if (p->q_rows < 0 || p->k_rows < 0 || p->q_rows > kMaxRows || p->k_rows > kMaxKeys || p->seqs < 1 ||
      p->seqs > (1 << 24) || p->q_heads < 1 || p->kv_heads < 1 || p->q_heads > 65535 ||
      p->q_heads % p->kv_heads != 0)
    return CUTBCE_ERR_SHAPE;
  if (p->head_dim < 8 || p->head_dim > 128 || p->head_dim % 8 != 0) return CUTBCE_ERR_UNSUPPORTED;
  if (!(p->scale == p->scale) || p->scale - p->scale != 0.f) return CUTBCE_ERR_SHAPE;
  const int64_t st[8] = {p->q_row_stride, p->q_head_stride, p->k_row_stride, p->k_head_stride,
                         p->v_row_stride, p->v_head_stride, p->k_seq_stride, p->v_seq_stride};
  for (int64_t s : st) {
    if (s < 0 || s > ((int64_t)1 << 40)) return CUTBCE_ERR_SHAPE;
    if (s * size_of(p->dtype) % 16 != 0) return CUTBCE_ERR_ALIGN;
  }
  // offsets inside a tile of up to 64 rows are 32-bit
  const int64_t row_max = (int64_t)1 << 22;
  if (st[0] > row_max || st[2] > row_max || st[4] > row_max || (int64_t)p->q_heads * p->head_dim > row_max)
    return CUTBCE_ERR_SHAPE;
  a->q_rs = st[0], a->q_hs = st[1], a->k_rs = st[2], a->k_hs = st[3], a->v_rs = st[4], a->v_hs = st[5];
  a->k_ss = st[6], a->v_ss = st[7];
  a->q_rows = p->q_rows, a->k_rows = p->k_rows;
  a->seqs = p->seqs, a->hq = p->q_heads, a->hk = p->kv_heads, a->group = p->q_heads / p->kv_heads;
  a->dh = p->head_dim, a->dtype = p->dtype, a->causal = p->causal != 0, a->scale = p->scale;
  a->cu_q = cu_q, a->cu_k = cu_k, a->k_lens = k_lens;
  a->q_pitch = p->q_rows / p->seqs, a->k_pitch = p->k_rows / p->seqs;
  if (cu_q && !cu_k && !k_lens) {  // self-attention: the keys' ranges are the queries'
    if (p->k_rows != p->q_rows) return CUTBCE_ERR_SHAPE;
    a->cu_k = cu_q;
  }
  return CUTBCE_OK;
}

}  // namespace

extern "C" {

cutbce_status cutbce_embedding_forward(int64_t n, int64_t vocab, int32_t dim, int32_t dtype, int32_t id_bytes,
                                       const void* ids, const void* table, float scale, void* out, void* stream) {
  cutbce_status s = check_embedding(n, vocab, dim, dtype);
  if (s != CUTBCE_OK) return s;
  if (id_bytes != 4 && id_bytes != 8) return CUTBCE_ERR_DTYPE;
  if (n == 0) return CUTBCE_OK;
  if (!ids || !table || !out) return CUTBCE_ERR_NULL;
  if (bad_align(ids, id_bytes) || bad_align(table, 16) || bad_align(out, 16)) return CUTBCE_ERR_ALIGN;
  return of_hip(launch_embedding_forward(n, vocab, dim, dtype, id_bytes, ids, table, scale, out, (hipStream_t)stream));
}

cutbce_status cutbce_embedding_backward_workspace_size(int64_t n, int64_t vocab, int32_t dim, int32_t dtype,
                                                       size_t* bytes) {
  cutbce_status s = check_embedding(n, vocab, dim, dtype);
  if (s != CUTBCE_OK) return s;
  if (n > kMaxSorted) return CUTBCE_ERR_SHAPE;
  if (!bytes) return CUTBCE_ERR_NULL;
  *bytes = embedding_backward_bytes(n, vocab, dim, dtype);
  return CUTBCE_OK;
}

cutbce_status cutbce_embedding_backward(int64_t n, int64_t vocab, int32_t dim, int32_t dtype, int32_t id_bytes,
                                        const void* ids, const void* dout, float scale, int32_t accumulate,
                                        void* dtable, void* workspace, size_t workspace_bytes, void* stream) {
  cutbce_status s = check_embedding(n, vocab, dim, dtype);
  if (s != CUTBCE_OK) return s;
  if (n > kMaxSorted) return CUTBCE_ERR_SHAPE;
  if (id_bytes != 4 && id_bytes != 8) return CUTBCE_ERR_DTYPE;
  if (!dtable || (n > 0 && (!ids || !dout || !workspace))) return CUTBCE_ERR_NULL;
  if (bad_align(ids, id_bytes) || bad_align(dout, 16) || bad_align(dtable, 16) || bad_align(workspace, 256))
    return CUTBCE_ERR_ALIGN;
  if (n > 0 && workspace_bytes < embedding_backward_bytes(n, vocab, dim, dtype)) return CUTBCE_ERR_WORKSPACE;
  return of_hip(launch_embedding_backward(n, vocab, dim, dtype, id_bytes, ids, dout, scale, accumulate != 0, dtable,
                                          (char*)workspace, (hipStream_t)stream));
}

cutbce_status cutbce_layer_norm_forward(int64_t rows, int32_t dim, int32_t dtype, int32_t param_dtype, const void* x,
                                        int64_t x_stride, const void* weight, const void* bias, float eps, void* y,
                                        float* mean, float* rstd, void* stream) {
  cutbce_status s = check_norm(rows, dim, dtype, param_dtype);
  if (s != CUTBCE_OK) return s;
  if (x_stride < dim || x_stride > ((int64_t)1 << 31) || !(eps >= 0.f)) return CUTBCE_ERR_SHAPE;
  if (rows == 0) return CUTBCE_OK;
  if (!x || !y || !mean != !rstd) return CUTBCE_ERR_NULL;
  const size_t e = size_of(dtype), pe = size_of(param_dtype);
  if (bad_align(x, e) || bad_align(y, e) || bad_align(weight, pe) || bad_align(bias, pe) || bad_align(mean, 4) ||
      bad_align(rstd, 4))
    return CUTBCE_ERR_ALIGN;
  return of_hip(launch_layer_norm_forward(rows, dim, dtype, param_dtype, x, x_stride, weight, bias, eps, y, mean, rstd,
                                          (hipStream_t)stream));
}

cutbce_status cutbce_layer_norm_backward_workspace_size(int64_t rows, int32_t dim, size_t* bytes) {
  cutbce_status s = check_norm(rows, dim, CUTBCE_F32, CUTBCE_F32);
  if (s != CUTBCE_OK) return s;
  if (!bytes) return CUTBCE_ERR_NULL;
  *bytes = layer_norm_backward_bytes(rows, dim);
  return CUTBCE_OK;
}

cutbce_status cutbce_layer_norm_backward(int64_t rows, int32_t dim, int32_t dtype, int32_t param_dtype,
                                         const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                         const void* weight, const float* mean, const float* rstd, void* dx,
                                         void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  cutbce_status s = check_norm(rows, dim, dtype, param_dtype);
  if (s != CUTBCE_OK) return s;
  if (x_stride < dim || x_stride > ((int64_t)1 << 31) || dy_stride < dim || dy_stride > ((int64_t)1 << 31))
    return CUTBCE_ERR_SHAPE;
  const bool params = dweight || dbias;
  if (rows > 0 && (!dy || !x || !mean || !rstd || (params && !workspace))) return CUTBCE_ERR_NULL;
  const size_t e = size_of(dtype), pe = size_of(param_dtype);
  if (bad_align(dy, e) || bad_align(x, e) || bad_align(dx, e) || bad_align(weight, pe) || bad_align(dweight, pe) ||
      bad_align(dbias, pe) || bad_align(mean, 4) || bad_align(rstd, 4) || bad_align(workspace, 256))
    return CUTBCE_ERR_ALIGN;
  if (rows > 0 && params && workspace_bytes < layer_norm_backward_bytes(rows, dim)) return CUTBCE_ERR_WORKSPACE;
  if (!dx && !params) return CUTBCE_OK;
  return of_hip(launch_layer_norm_backward(rows, dim, dtype, param_dtype, dy, dy_stride, x, x_stride, weight, mean,
                                           rstd, dx, dweight, dbias, (char*)workspace, (hipStream_t)stream));
}

cutbce_status cutbce_attention_workspace_size(const cutbce_attention* p, int32_t backward, size_t* bytes) {
  Attn a = {};
  // (without the ranges' arrays the sizes may be those of single tokens over a cache, which take the most)
  cutbce_status s = make_attn(p, nullptr, nullptr, nullptr, &a);
  if (s != CUTBCE_OK) return s;
  if (!attention_fits(a, backward != 0)) return CUTBCE_ERR_SHAPE;
  if (!bytes) return CUTBCE_ERR_NULL;
  *bytes = attention_bytes(a, backward != 0);
  return CUTBCE_OK;
}

cutbce_status cutbce_attention_forward(const cutbce_attention* p, const void* q, const void* k, const void* v,
                                       const int32_t* cu_q, const int32_t* cu_k, const int32_t* k_lens, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  Attn a = {};
  cutbce_status s = make_attn(p, cu_q, cu_k, k_lens, &a);
  if (s != CUTBCE_OK) return s;
  if (!attention_fits(a, false)) return CUTBCE_ERR_SHAPE;
  if (a.q_rows == 0) return CUTBCE_OK;
  const size_t need = attention_bytes(a, false);
  if (!q || !out || (a.k_rows > 0 && (!k || !v)) || (need && !workspace)) return CUTBCE_ERR_NULL;
  if (bad_align(q, 16) || bad_align(k, 16) || bad_align(v, 16) || bad_align(out, 16) || bad_align(cu_q, 4) ||
      bad_align(cu_k, 4) || bad_align(k_lens, 4) || bad_align(lse, 4) || bad_align(workspace, 256))
    return CUTBCE_ERR_ALIGN;
  if (workspace_bytes < need) return CUTBCE_ERR_WORKSPACE;
  a.q = q, a.k = k, a.v = v;
  return of_hip(launch_attention_forward(a, out, lse, (char*)workspace, (hipStream_t)stream));
}

cutbce_status cutbce_attention_backward(const cutbce_attention* p, const void* dout, const void* q, const void* k,
                                        const void* v, const void* out, const float* lse, const int32_t* cu_q,
                                        const int32_t* cu_k, const int32_t* k_lens, void* dq, void* dk, void* dv,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  Attn a = {};
  cutbce_status s = make_attn(p, cu_q, cu_k, k_lens, &a);
  if (s != CUTBCE_OK) return s;
  if (!attention_fits(a, true)) return CUTBCE_ERR_SHAPE;
  if (a.q_rows == 0 && a.k_rows == 0) return CUTBCE_OK;
  const size_t need = attention_bytes(a, true);
  if ((a.q_rows > 0 && (!dout || !q || !out || !lse || !dq)) || (a.k_rows > 0 && (!k || !v || !dk || !dv)) ||
      (need && !workspace))
    return CUTBCE_ERR_NULL;
  if (bad_align(dout, 16) || bad_align(q, 16) || bad_align(k, 16) || bad_align(v, 16) || bad_align(out, 16) ||
      bad_align(dq, 16) || bad_align(dk, 16) || bad_align(dv, 16) || bad_align(cu_q, 4) || bad_align(cu_k, 4) ||
      bad_align(k_lens, 4) || bad_align(lse, 4) || bad_align(workspace, 256))
    return CUTBCE_ERR_ALIGN;
  if (workspace_bytes < need) return CUTBCE_ERR_WORKSPACE;
  a.q = q, a.k = k, a.v = v;
  return of_hip(launch_attention_backward(a, dout, out, lse, dq, dk, dv, (char*)workspace, (hipStream_t)stream));
}

}  // extern "C"
