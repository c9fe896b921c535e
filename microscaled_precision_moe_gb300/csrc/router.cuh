// Launchers of the router: top-k choice, routing weights, expert counts and
// balance loss, and their gradient.
#pragma once
#include "common.cuh"

namespace mpm {

struct RouteArgs {
  const void* logits; int bf16; long long T; int E; long long ld; int k;
  int sigmoid, normalize; float scale;
  const float* bias;                       // [E], choice only (nullable)
  const uint8_t* mask;                     // [T], 0 = a token that does not count (nullable)
  // forward
  int* ids; float* prob;                   // [T, k]
  int* counts; float* load;                // [E]
  int* n_tokens; float* loss;              // [1]
  float* ws_load; int* ws_counts; int* ws_n;   // [parts, E], [parts, E], [parts]
  // backward
  const int* in_ids; const int* in_counts; const int* in_n;
  const float* dprob; const float* dloss;  // [T, k], [1] (nullable)
  void* dlogits; long long ldd; int out_bf16;
  int* status;
  int vec, vec_out, cluster;               // set by the launchers: rows read and written by
                                           // words; one cluster routes everything
};
size_t route_ws_bytes(long long T, int E);
cudaError_t launch_route(const RouteArgs& a, void* ws, cudaStream_t st);
cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t st);

}  // namespace mpm
