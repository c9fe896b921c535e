// Launchers of the residual RMSNorm, forward (with MXFP8 output) and backward.
#pragma once
#include "common.cuh"

namespace mpm {

struct NormFwd {
  const uint16_t* x; long long ldx;        // bf16 [M, K]
  const uint16_t* r; long long ldr;        // residual, bf16 [M, K] (nullable)
  const void* w; int w_f32;                // weight [K], bf16 or fp32
  float eps;
  uint16_t* h; long long ldh;              // x + r, bf16 (nullable)
  uint16_t* y; long long ldy;              // bf16 (nullable)
  float* rstd;                             // fp32 [M] (nullable)
  uint8_t* q; uint8_t* s; long long s_cols_pad;   // MXFP8 row copy of y (nullable)
  long long M; int K; float rk;            // rk = 1 / K
};
cudaError_t launch_add_rmsnorm(const NormFwd& p, cudaStream_t st);

struct NormBwd {
  const uint16_t* dy; long long lddy;
  const uint16_t* dy2; long long lddy2;    // second gradient of y (nullable)
  const uint16_t* h; long long ldh;
  const void* w; int w_f32;
  const float* rstd;
  const uint16_t* dh; long long lddh;      // gradient arriving on h itself (nullable)
  uint16_t* dx; long long lddx;
  float* dw;                               // fp32 [K] (nullable)
  float* part;                             // workspace [parts, K]
  int* status;
  long long M; int K;
};
long long rmsnorm_backward_parts(long long M, int K);
cudaError_t launch_add_rmsnorm_backward(const NormBwd& p, cudaStream_t st);

}  // namespace mpm
