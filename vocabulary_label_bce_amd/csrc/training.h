// Launchers of the training step's operators (softmax cross entropy, gradient norm, AdamW) that training_api.hip calls.
#pragma once
#include "encoder.h"

namespace cutbce {

// ---------------------------------------------------------------------------------------------------------
// Lists of tensors. A launch takes kListed of them by value, as kernel arguments: nothing is copied to the device
// first. ---------------------------------------------------------------------------------------------------------
constexpr int kListed = 48;
constexpr int kChunk = 4096;  // elements of a workgroup
constexpr int kBlock8 = 256;  // elements that share a scale in states of 8 bits: 16 lanes' sixteen each

struct AdamEntry {
  void *p, *m, *v;
  const void* g;
  float *ms, *vs;  // scales of the states' blocks (8 bits)
  float* master;   // float32 copy of p, or NULL
  int64_t n;
  float decay;
  int16_t p_type, g_type;
};
struct AdamHow {
  int32_t* step;
  const float *lr_at, *norm;
  float lr, beta1, beta2, eps, max_norm;
  float rest1, rest2;  // 1 - beta, formed in float64
  float log_beta1, log_beta2;
  uint32_t seed;
};
struct AdamArgs {
  AdamEntry e[kListed];
  uint32_t start[kListed];  // first workgroup of each; 0xffffffff behind the last
  AdamHow how;
  uint32_t first;  // number of the first tensor
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");
hipError_t launch_adamw(const AdamArgs& a, unsigned blocks, bool bits8, hipStream_t st);
hipError_t launch_step(int32_t* step, hipStream_t st);

constexpr int kNormListed = 128;
constexpr int kNormChunk = 16384;
struct NormArgs {
  const void* g[kNormListed];
  int64_t n[kNormListed];
  uint32_t start[kNormListed];
  uint8_t type[kNormListed];
  double* partials;  // of this launch's workgroups
};
static_assert(sizeof(NormArgs) <= 4096, "kernel arguments");
hipError_t launch_norm(const NormArgs& a, unsigned blocks, hipStream_t st);
hipError_t launch_norm_join(const double* partials, int64_t n, float* norm, hipStream_t st);

// ---------------------------------------------------------------------------------------------------------
// Softmax cross entropy: z = scale H E^T, rows with a target in [0, V) counted ("compact") 0 .. n - 1 in their order.
// ---------------------------------------------------------------------------------------------------------
constexpr int64_t kCeMaxRows = (int64_t)1 << 20;
constexpr int kCeMaxDim = 16384;

struct CeHead {
  int32_t n;     // rows that have a target
  float weight;  // sum of their weights
};

// What the forward leaves for the backward, as byte offsets into `saved`; arrays of R entries unless said. What a row
// brings to dz: exp2(c z - shift), or at its target `own` instead; coef = w / W.
struct CeSaved {
  size_t head, rows, place, target, shift, own, coef, hc, dh, bytes;
};
struct Ce {
  int64_t R, V;
  int D, dtype;
  float scale;
  const void* E;
  CeSaved at;
  char* saved;
  char* ws;
};
// The sweeps of narrow rows (softmax_sweep.hip): the sums of all rows, with their dH in `saved` where grad, and the
// backward.
bool ce_swept(int D, int dtype);  // whether they take this problem
size_t ce_rows_bytes(int64_t R, int D, bool grad);
hipError_t launch_ce_rows(const Ce& c, char* ws, bool grad, const float* zt, float* row_loss, float* each,
                          hipStream_t st);
size_t ce_items_bytes(int D);
hipError_t launch_ce_items(const Ce& c, char* ws, const float* grad, void* dH, void* dE, hipStream_t st);
CeSaved ce_saved(int64_t R, int64_t V, int D, int dtype);
size_t ce_forward_bytes(int64_t R, int64_t V, int D, int dtype, bool want_grad);
size_t ce_backward_bytes(int64_t R, int64_t V, int D, int dtype);
hipError_t launch_ce_forward(const Ce& c, int id_bytes, const void* H, const void* targets, const float* weight,
                             bool want_grad, float* loss, float* row_loss, hipStream_t st);
hipError_t launch_ce_backward(const Ce& c, const float* grad, void* dH, void* dE, hipStream_t st);

}  // namespace cutbce
