// Launchers of the token log probabilities and of their gradient.
#pragma once
#include "common.cuh"

namespace mpm {

struct LogprobFwd {
  const void* logits; int f32; long long T, V, ld;
  const void* targets; int targets_i64;    // [T] (nullable: every row counts, no logp)
  float inv_t;                             // 1 / temperature
  int top;
  float* logp;                             // [T] (nullable without targets)
  float* lse;                              // [T]
  float* entropy;                          // [T] (nullable)
  int* top_ids; float* top_logp;           // [T, top]
  int* status;
};
cudaError_t launch_token_logprob(const LogprobFwd& p, cudaStream_t st);

struct LogprobBwd {
  const void* logits; int f32; long long T, V, ld;
  const void* targets; int targets_i64;    // [T] (nullable)
  const float* lse;                        // [T]
  const float* logp;                       // [T] (nullable: log p of the targets from lse)
  const float* dlogp;                      // [T] (nullable)
  const float* entropy; const float* dentropy;   // [T] (nullable, both or none)
  float inv_t; float zero;                 // 1 / temperature; 0
  void* out; int out_f32; long long ldo;
  int* status;
};
cudaError_t launch_token_logprob_backward(const LogprobBwd& p, cudaStream_t st);

}  // namespace mpm
