// Residual addition and root-mean-square norm for sm_103a, with the MXFP8 copy
// of the result that the block-scaled GEMMs read, and their gradient.
//
//   h = x + r,  rstd = (mean_K h^2 + eps)^(-1/2),  y = h rstd w
//
// The sum and its square mean are held in fp32; h and y are rounded to bf16
// once, each from its fp32 value.  The 8-bit output is the quantisation of the
// bf16 y, not of its fp32 value, so that it holds the bytes mpm_mxfp8_quantize
// makes of y: a rollout that reads these codes and a training step that
// quantises the stored y then run on the same operands.
//
// A row is held in the registers of the threads of one block (VEC consecutive
// elements per load, IT loads per thread), so every operand is read once.
#include "norm.cuh"
#include "mxfp8.cuh"

namespace mpm {

constexpr int kNormMaxThreads = 512;

MPM_DEV float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
MPM_DEV uint16_t f_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <int VEC>
MPM_DEV void load_bf16(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[2 * j] = bf16lo(w[j]); v[2 * j + 1] = bf16hi(w[j]); }
  } else {
    v[0] = bf16_f(*p);
  }
}
template <int VEC>
MPM_DEV void store_bf16(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (uint32_t)f_bf16(v[2 * j]) | ((uint32_t)f_bf16(v[2 * j + 1]) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *p = f_bf16(v[0]);
  }
}
template <int VEC>
MPM_DEV void load_weight(const void* w, int f32, int k, float (&v)[VEC]) {
  if (f32) {
    const float* p = static_cast<const float*>(w) + k;
    if constexpr (VEC == 8) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      v[0] = *p;
    }
  } else {
    load_bf16<VEC>(static_cast<const uint16_t*>(w) + k, v);
  }
}

// sum over the block's threads, in a fixed order; every thread gets it
MPM_DEV float block_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  const int nw = blockDim.x >> 5;
  __syncthreads();                       // sh free (an earlier call's reads are over)
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < nw; ++i) t = __fadd_rn(t, sh[i]);
  return t;
}

template <int VEC, int IT>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_kernel(const NormFwd p) {
  __shared__ float sh[kNormMaxThreads / 32];
  const long long row = blockIdx.x;
  const int t = threadIdx.x, nt = blockDim.x;
  const int nblk = p.K >> 5;
  if (row >= p.M) {                      // padding rows of the last scale tile
    for (int c = t; c < (int)p.s_cols_pad; c += nt) p.s[sf_offset(row, c, p.s_cols_pad)] = 0;
    return;
  }
  float h[IT][VEC];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * nt + t) * VEC;
    if (k < p.K) {
      load_bf16<VEC>(p.x + row * p.ldx + k, h[i]);
      if (p.r) {
        float r[VEC];
        load_bf16<VEC>(p.r + row * p.ldr + k, r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[i][j] = __fadd_rn(h[i][j], r[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) ss = __fmaf_rn(h[i][j], h[i][j], ss);
  }
  ss = block_sum(ss, sh);
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)p.K), p.eps));
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * nt + t) * VEC;
    const bool in = k < p.K;
    float y[VEC];
    if (in) {
      if (p.h) store_bf16<VEC>(p.h + row * p.ldh + k, h[i]);
      load_weight<VEC>(p.w, p.w_f32, k, y);
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[j] = __fmul_rn(__fmul_rn(h[i][j], rstd), y[j]);
      if (p.y) store_bf16<VEC>(p.y + row * p.ldy + k, y);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[j] = 0.0f;
    }
    if (p.q) {
      // K % 32 == 0: a block of 32 lies in 32 / VEC neighbouring lanes
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < VEC; ++j) m = max(m, (uint32_t)f_bf16(y[j]) & 0x7FFFu);
#pragma unroll
      for (int o = 16 / VEC; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const int e = mx_exponent(m << 16);
      if (in) {
        const uint64_t sc = f32x2_splat(pow2_neg(e));
        uint8_t* dst = p.q + row * (long long)p.K + k;
        if constexpr (VEC == 8) {
          uint32_t c[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            c[j] = e4m3x2_scaled((uint32_t)f_bf16(y[2 * j]) | ((uint32_t)f_bf16(y[2 * j + 1]) << 16), sc);
          *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        } else {
          *dst = (uint8_t)e4m3x2_scaled(f_bf16(y[0]), sc);
        }
        if (k % 32 == 0) p.s[sf_offset(row, k >> 5, p.s_cols_pad)] = (uint8_t)(e + 127);
      }
    }
  }
  if (p.q && t < (int)p.s_cols_pad - nblk) p.s[sf_offset(row, nblk + t, p.s_cols_pad)] = 0;
}

// ---------------------------------------------------------------- backward
// With xh = h rstd and g = dy w:
//   dx = rstd (g - xh mean_K(g xh)) + dh,   dw = sum over rows of dy xh.
// Blocks walk the rows blockIdx.x, blockIdx.x + gridDim.x, ...; each keeps its
// columns' share of dw in fp32 registers and writes it to its row of the
// workspace, which a second kernel sums in row order (no atomics: the same
// bytes every time).
template <int VEC, int IT>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_bwd_kernel(const NormBwd p) {
  __shared__ float sh[kNormMaxThreads / 32];
  const int t = threadIdx.x, nt = blockDim.x;
  float dw[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = 0.0f;
  for (long long row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float rstd = p.rstd[row];
    float g[IT][VEC], xh[IT][VEC];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = (i * nt + t) * VEC;
      if (k < p.K) {
        load_bf16<VEC>(p.dy + row * p.lddy + k, g[i]);
        if (p.dy2) {
          float d[VEC];
          load_bf16<VEC>(p.dy2 + row * p.lddy2 + k, d);
#pragma unroll
          for (int j = 0; j < VEC; ++j) g[i][j] = __fadd_rn(g[i][j], d[j]);
        }
        load_bf16<VEC>(p.h + row * p.ldh + k, xh[i]);
        float w[VEC];
        load_weight<VEC>(p.w, p.w_f32, k, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] = __fmul_rn(xh[i][j], rstd);
          dw[i][j] = __fmaf_rn(g[i][j], xh[i][j], dw[i][j]);
          g[i][j] = __fmul_rn(g[i][j], w[j]);
          c = __fmaf_rn(g[i][j], xh[i][j], c);
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[i][j] = xh[i][j] = 0.0f;
      }
    }
    c = __fdiv_rn(block_sum(c, sh), (float)p.K);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = (i * nt + t) * VEC;
      if (k >= p.K) continue;
      float d[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] = __fmul_rn(rstd, __fmaf_rn(-xh[i][j], c, g[i][j]));
      if (p.dh) {
        float v[VEC];
        load_bf16<VEC>(p.dh + row * p.lddh + k, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = __fadd_rn(d[j], v[j]);
      }
      store_bf16<VEC>(p.dx + row * p.lddx + k, d);
    }
  }
  if (!p.dw) return;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * nt + t) * VEC;
    if (k >= p.K) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) p.part[(long long)blockIdx.x * p.K + k + j] = dw[i][j];
  }
}

__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float* part, int parts, int K, float* dw) {
  const int k = blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= K) return;
  float s = 0.0f;
  for (int i = 0; i < parts; ++i) s = __fadd_rn(s, part[(long long)i * K + k]);
  dw[k] = s;
}

// ---------------------------------------------------------------- launchers
static bool vec8(const void* p, long long ld) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0);
}
static unsigned norm_threads(int K, int per_thread) {
  const int n = (K + per_thread - 1) / per_thread;
  return (unsigned)((n + 31) / 32 * 32);
}

cudaError_t launch_add_rmsnorm(const NormFwd& p, cudaStream_t st) {
  const long long rows = p.q ? (p.M + 127) / 128 * 128 : p.M;
  const bool v = p.K % 8 == 0 && vec8(p.x, p.ldx) && vec8(p.r, p.ldr) && vec8(p.h, p.ldh) &&
                 vec8(p.y, p.ldy) && vec8(p.w, 0);
  const dim3 grid((unsigned)rows);
  if (v) {
    if (p.K <= 8 * kNormMaxThreads) add_rmsnorm_kernel<8, 1><<<grid, norm_threads(p.K, 8), 0, st>>>(p);
    else add_rmsnorm_kernel<8, 4><<<grid, norm_threads(p.K, 32), 0, st>>>(p);
  } else {
    if (p.K <= 4 * kNormMaxThreads) add_rmsnorm_kernel<1, 4><<<grid, norm_threads(p.K, 4), 0, st>>>(p);
    else add_rmsnorm_kernel<1, 32><<<grid, norm_threads(p.K, 32), 0, st>>>(p);
  }
  return cudaGetLastError();
}

// blocks of the backward: enough to fill 152 SMs, each with its own partial dw
long long rmsnorm_backward_parts(long long M, int) { return M < 304 ? M : 304; }

cudaError_t launch_add_rmsnorm_backward(const NormBwd& p, cudaStream_t st) {
  const bool v = p.K % 8 == 0 && vec8(p.dy, p.lddy) && vec8(p.dy2, p.lddy2) && vec8(p.h, p.ldh) &&
                 vec8(p.dh, p.lddh) && vec8(p.dx, p.lddx) && vec8(p.w, 0);
  const int parts = (int)rmsnorm_backward_parts(p.M, p.K);
  if (v) {
    if (p.K <= 8 * kNormMaxThreads) add_rmsnorm_bwd_kernel<8, 1><<<parts, norm_threads(p.K, 8), 0, st>>>(p);
    else add_rmsnorm_bwd_kernel<8, 4><<<parts, norm_threads(p.K, 32), 0, st>>>(p);
  } else {
    if (p.K <= 4 * kNormMaxThreads) add_rmsnorm_bwd_kernel<1, 4><<<parts, norm_threads(p.K, 4), 0, st>>>(p);
    else add_rmsnorm_bwd_kernel<1, 32><<<parts, norm_threads(p.K, 32), 0, st>>>(p);
  }
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !p.dw) return err;
  rmsnorm_dw_kernel<<<(unsigned)((p.K + 255) / 256), 256, 0, st>>>(p.part, parts, p.K, p.dw);
  return cudaGetLastError();
}

}  // namespace mpm
