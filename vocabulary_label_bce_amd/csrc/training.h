// Launchers of the training step's operators (softmax cross entropy, gradient norm, AdamW) that training_api.hip calls.
#pragma once
#include "encoder.h"

namespace cutbce {

// ---------------------------------------------------------------------------------------------------------
// Lists of tensors. A launch takes kListed of them by value, as kernel arguments: nothing is copied to the device first.
// ---------------------------------------------------------------------------------------------------------
constexpr int kListed = 48;
constexpr int kChunk = 4096;  // elements of a workgroup
constexpr int kBlock8 = 256;  // elements that share a scale in states of 8 bits: a wave's four each

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

}  // namespace cutbce
