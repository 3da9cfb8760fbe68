// C ABI of the training step's operators (declared in include/cutbce.h): argument checks and launches.
#include <math.h>

#include "../../include/cutbce.h"
#include "training.h"

using namespace cutbce;

namespace {

bool bad_align(const void* p, size_t a) { return p && ((uintptr_t)p % a) != 0; }
bool known(int dtype) { return dtype == CUTBCE_F32 || dtype == CUTBCE_BF16; }
size_t size_of(int dtype) { return dtype == CUTBCE_BF16 ? 2 : 4; }
cutbce_status of_hip(hipError_t e) { return e == hipSuccess ? CUTBCE_OK : CUTBCE_ERR_HIP; }

constexpr int kMaxTensors = 1 << 20;
constexpr int64_t kMaxChunks = 0x7fffffff;

// Workgroups of all tensors, or -1 where there are too many.
int64_t chunks_of(int32_t count, const int64_t* n, int64_t chunk) {
  int64_t sum = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (n[i] < 0 || n[i] > kMaxChunks * chunk) return -1;
    sum += (n[i] + chunk - 1) / chunk;
    if (sum + count > kMaxChunks) return -1;
  }
  return sum;
}

constexpr int64_t kMaxVocab = (int64_t)0x7fffffff - 1024;

cutbce_status check_ce(int64_t rows, int64_t vocab, int32_t dim, int32_t dtype) {
  if (!known(dtype)) return CUTBCE_ERR_DTYPE;
  if (rows < 0 || rows > kCeMaxRows || vocab < 1 || vocab > kMaxVocab) return CUTBCE_ERR_SHAPE;
  if (dim < 8 || dim > kCeMaxDim || dim % 8 != 0) return CUTBCE_ERR_UNSUPPORTED;
  return CUTBCE_OK;
}

}  // namespace

extern "C" {

cutbce_status cutbce_cross_entropy_saved_size(int64_t rows, int64_t vocab, int32_t dim, int32_t dtype, size_t* bytes) {
  if (!bytes) return CUTBCE_ERR_NULL;
  const cutbce_status s = check_ce(rows, vocab, dim, dtype);
  if (s == CUTBCE_OK) *bytes = ce_saved(rows, vocab, dim, dtype).bytes;
  return s;
}

cutbce_status cutbce_cross_entropy_workspace_size(int64_t rows, int64_t vocab, int32_t dim, int32_t dtype,
                                                  int32_t which, size_t* bytes) {
  if (!bytes) return CUTBCE_ERR_NULL;
  const cutbce_status s = check_ce(rows, vocab, dim, dtype);
  if (s != CUTBCE_OK) return s;
  if (which < 0 || which > 2) return CUTBCE_ERR_SHAPE;
  *bytes = which == 2 ? ce_backward_bytes(rows, vocab, dim, dtype)
                      : ce_forward_bytes(rows, vocab, dim, dtype, which == 1);
  return CUTBCE_OK;
}

cutbce_status cutbce_cross_entropy_forward(int64_t rows, int64_t vocab, int32_t dim, int32_t dtype, int32_t id_bytes,
                                           const void* H, const void* E, const void* targets, const float* row_weight,
                                           float scale, float* loss, float* row_loss, void* saved, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  const cutbce_status s = check_ce(rows, vocab, dim, dtype);
  if (s != CUTBCE_OK) return s;
  if (id_bytes != 4 && id_bytes != 8) return CUTBCE_ERR_DTYPE;
  if (!(fabsf(scale) < INFINITY)) return CUTBCE_ERR_SHAPE;
  const size_t need = ce_forward_bytes(rows, vocab, dim, dtype, saved != nullptr);
  if (!E || !loss || (need && !workspace) || (rows > 0 && (!H || !targets))) return CUTBCE_ERR_NULL;
  if (bad_align(H, 16) || bad_align(E, 16) || bad_align(targets, id_bytes) || bad_align(row_weight, 4) ||
      bad_align(loss, 4) || bad_align(row_loss, 4) || bad_align(saved, 256) || bad_align(workspace, 256))
    return CUTBCE_ERR_ALIGN;
  if (workspace_bytes < need) return CUTBCE_ERR_WORKSPACE;
  Ce c = {rows, vocab, dim, dtype, scale, E, ce_saved(rows, vocab, dim, dtype), (char*)saved, (char*)workspace};
  if (!saved) c.saved = c.ws + need - c.at.bytes;
  return of_hip(launch_ce_forward(c, id_bytes, H, targets, row_weight, saved != nullptr, loss, row_loss,
                                  (hipStream_t)stream));
}

cutbce_status cutbce_cross_entropy_backward(int64_t rows, int64_t vocab, int32_t dim, int32_t dtype, const void* E,
                                            float scale, const float* grad_loss, const void* saved, void* dH, void* dE,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  const cutbce_status s = check_ce(rows, vocab, dim, dtype);
  if (s != CUTBCE_OK) return s;
  if (!(fabsf(scale) < INFINITY)) return CUTBCE_ERR_SHAPE;
  const size_t need = ce_backward_bytes(rows, vocab, dim, dtype);
  if (!E || !grad_loss || !saved || (need && !workspace)) return CUTBCE_ERR_NULL;
  if (bad_align(E, 16) || bad_align(grad_loss, 4) || bad_align(saved, 256) || bad_align(dH, 16) || bad_align(dE, 16) ||
      bad_align(workspace, 256))
    return CUTBCE_ERR_ALIGN;
  if (workspace_bytes < need) return CUTBCE_ERR_WORKSPACE;
  if (!dH && !dE) return CUTBCE_OK;
  const Ce c = {rows, vocab, dim, dtype, scale, E, ce_saved(rows, vocab, dim, dtype), (char*)saved, (char*)workspace};
  return of_hip(launch_ce_backward(c, grad_loss, dH, dE, (hipStream_t)stream));
}

cutbce_status cutbce_grad_norm_workspace_size(int32_t count, const int64_t* n, size_t* bytes) {
  if (!bytes || (count > 0 && !n)) return CUTBCE_ERR_NULL;
  if (count < 0 || count > kMaxTensors) return CUTBCE_ERR_SHAPE;
  const int64_t chunks = chunks_of(count, n, kNormChunk);
  if (chunks < 0) return CUTBCE_ERR_SHAPE;
  *bytes = ((size_t)chunks * sizeof(double) + 255) / 256 * 256;
  return CUTBCE_OK;
}

cutbce_status cutbce_grad_norm(int32_t count, const void* const* grads, const int64_t* n, const int32_t* dtypes,
                               float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (count > 0 && (!grads || !n || !dtypes)) return CUTBCE_ERR_NULL;
  size_t need = 0;
  const cutbce_status s = cutbce_grad_norm_workspace_size(count, n, &need);
  if (s != CUTBCE_OK) return s;
  for (int32_t i = 0; i < count; ++i) {
    if (!known(dtypes[i])) return CUTBCE_ERR_DTYPE;
    if (n[i] > 0 && !grads[i]) return CUTBCE_ERR_NULL;
    if (bad_align(grads[i], size_of(dtypes[i]))) return CUTBCE_ERR_ALIGN;
  }
  if (!norm || (need && !workspace)) return CUTBCE_ERR_NULL;
  if (bad_align(norm, 4) || bad_align(workspace, 256)) return CUTBCE_ERR_ALIGN;
  if (workspace_bytes < need) return CUTBCE_ERR_WORKSPACE;
  double* partials = (double*)workspace;
  const hipStream_t st = (hipStream_t)stream;
  int64_t done = 0;  // workgroups of earlier launches
  NormArgs a;
  int listed = 0;
  int64_t blocks = 0;
  auto launch = [&]() -> hipError_t {
    for (int k = listed; k < kNormListed; ++k) a.start[k] = 0xffffffffu;
    a.partials = partials + done;
    const hipError_t e = launch_norm(a, (unsigned)blocks, st);
    done += blocks, listed = 0, blocks = 0;
    return e;
  };
  for (int32_t i = 0; i < count; ++i) {
    // a tensor of more workgroups than a launch takes goes in turns, from a later element each
    for (int64_t from = 0; from < n[i];) {
      const int64_t want = (n[i] - from + kNormChunk - 1) / kNormChunk, room = kMaxGrid - blocks;
      const int64_t part = want < room ? want : room;
      a.g[listed] = (const char*)grads[i] + from * size_of(dtypes[i]);
      a.n[listed] = n[i] - from < part * kNormChunk ? n[i] - from : part * kNormChunk;
      a.start[listed] = (uint32_t)blocks;
      a.type[listed] = (uint8_t)dtypes[i];
      ++listed, blocks += part, from += part * kNormChunk;
      if (listed == kNormListed || blocks == kMaxGrid) {
        const hipError_t e = launch();
        if (e != hipSuccess) return CUTBCE_ERR_HIP;
      }
    }
  }
  if (listed) {
    const hipError_t e = launch();
    if (e != hipSuccess) return CUTBCE_ERR_HIP;
  }
  return of_hip(launch_norm_join(partials, done, norm, st));
}

cutbce_status cutbce_adamw_step(const cutbce_adamw_tensors* x, const cutbce_adamw* how, void* stream) {
  if (!how || !x || !how->step) return CUTBCE_ERR_NULL;
  if (x->count < 0 || x->count > kMaxTensors) return CUTBCE_ERR_SHAPE;
  if (how->state_bits != 32 && how->state_bits != 8) return CUTBCE_ERR_DTYPE;
  if (bad_align(how->step, 4) || bad_align(how->lr_at, 4) || bad_align(how->norm, 4)) return CUTBCE_ERR_ALIGN;
  if (!(how->beta1 >= 0 && how->beta1 < 1 && how->beta2 >= 0 && how->beta2 < 1) ||
      !(how->eps >= 0 && how->eps < INFINITY) || (!how->lr_at && !(fabs(how->lr) < INFINITY)) ||
      (how->norm && !(how->max_norm >= 0)))
    return CUTBCE_ERR_SHAPE;
  const bool b8 = how->state_bits == 8;
  const int32_t count = x->count;
  if (count > 0 && (!x->param || !x->grad || !x->exp_avg || !x->exp_avg_sq || !x->n || !x->param_dtype ||
                    !x->grad_dtype || !x->weight_decay || (b8 && (!x->exp_avg_scale || !x->exp_avg_sq_scale))))
    return CUTBCE_ERR_NULL;
  for (int32_t i = 0; i < count; ++i) {
    const int64_t n = x->n[i];
    const void *p = x->param[i], *g = x->grad[i], *m = x->exp_avg[i], *v = x->exp_avg_sq[i];
    if (!known(x->param_dtype[i]) || !known(x->grad_dtype[i])) return CUTBCE_ERR_DTYPE;
    if (n < 0 || n > kMaxGrid * kChunk || !(fabsf(x->weight_decay[i]) < INFINITY)) return CUTBCE_ERR_SHAPE;
    if (n == 0) continue;
    if (!p || !g || !m || !v || (b8 && (!x->exp_avg_scale[i] || !x->exp_avg_sq_scale[i]))) return CUTBCE_ERR_NULL;
    if (bad_align(p, size_of(x->param_dtype[i])) || bad_align(g, size_of(x->grad_dtype[i])) ||
        (!b8 && (bad_align(m, 4) || bad_align(v, 4))) ||
        (b8 && (bad_align(x->exp_avg_scale[i], 4) || bad_align(x->exp_avg_sq_scale[i], 4))) ||
        (x->master && bad_align(x->master[i], 4)))
      return CUTBCE_ERR_ALIGN;
  }
  const hipStream_t st = (hipStream_t)stream;
  AdamArgs a;
  a.how.step = how->step, a.how.lr_at = how->lr_at, a.how.norm = how->norm;
  a.how.lr = (float)how->lr, a.how.eps = (float)how->eps, a.how.max_norm = (float)how->max_norm;
  a.how.beta1 = (float)how->beta1, a.how.beta2 = (float)how->beta2;
  a.how.rest1 = (float)(1 - how->beta1), a.how.rest2 = (float)(1 - how->beta2);
  a.how.log_beta1 = (float)log(how->beta1), a.how.log_beta2 = (float)log(how->beta2);
  a.how.seed = how->seed;
  int listed = 0;
  int64_t blocks = 0;
  for (int32_t i = 0; i < count; ++i) {
    const int64_t want = (x->n[i] + kChunk - 1) / kChunk;
    if (listed && (listed == kListed || blocks + want > kMaxGrid)) {
      for (int k = listed; k < kListed; ++k) a.start[k] = 0xffffffffu;
      if (blocks && launch_adamw(a, (unsigned)blocks, b8, st) != hipSuccess) return CUTBCE_ERR_HIP;
      listed = 0, blocks = 0;
    }
    if (!listed) a.first = (uint32_t)i;
    a.e[listed] = {x->param[i], x->exp_avg[i], x->exp_avg_sq[i], x->grad[i], b8 ? (float*)x->exp_avg_scale[i] : nullptr,
                   b8 ? (float*)x->exp_avg_sq_scale[i] : nullptr, x->master ? (float*)x->master[i] : nullptr, x->n[i],
                   x->weight_decay[i], (int16_t)x->param_dtype[i], (int16_t)x->grad_dtype[i]};
    a.start[listed] = (uint32_t)blocks;
    ++listed, blocks += want;
  }
  if (blocks) {
    for (int k = listed; k < kListed; ++k) a.start[k] = 0xffffffffu;
    if (launch_adamw(a, (unsigned)blocks, b8, st) != hipSuccess) return CUTBCE_ERR_HIP;
  }
  return of_hip(launch_step(how->step, st));
}

}  // extern "C"
