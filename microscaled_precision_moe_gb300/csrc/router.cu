// Router of the expert layer for sm_103a: the k experts of each token, their
// weights, the tokens each expert receives and the balance loss, and the
// gradient with respect to the logits.
//
// A logit that is NaN or at or below bf16's lowest finite value (so -inf, and
// both types' lowest values, which masks use) takes an expert out of reach: its
// score is 0, it is chosen only where fewer than k are left (its weight is then
// 0), and it is never counted.  +inf reads as the largest finite value.
//   softmax:  s_e = exp(l_e - max) / sum,     chosen by l_e
//   sigmoid:  s_e = 1 / (1 + exp(-l_e)),      chosen by s_e + bias_e
// weights w_j = s of the j-th choice, over their sum if `normalize`, times
// `scale`; a masked token's weights are 0 and it is not counted.  With n
// unmasked tokens, c_e the counts and P_e the mean over them of a token's
// scores as shares of one, loss = E / (k n) sum_e c_e P_e: 1 at perfect balance.
//
// One warp per token, expert e in lane e % 32.  The choice compares the keys
// themselves (order-preserving integers), k times the warp's maximum and the
// lowest expert that holds it, so it is exact and ties go to the lower expert.
// Scores use expf and IEEE division: with a bias the choice depends on their
// last bit.  Sums over tokens go through per-block partials added in a fixed
// order (no floating-point atomics).
#include "router.cuh"

namespace mpm {

constexpr int kRouteWarps = 8;
constexpr int kRouteMaxParts = 608;
constexpr float kDeadLogit = -3.3895313892515355e38f;   // bf16's lowest finite value
constexpr float kLargest = 3.4028234663852886e38f;

// order-preserving map of a number (not NaN) to an integer above 0
MPM_DEV uint32_t ordered_bits(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));      // -0 compares equal to +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

MPM_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
MPM_DEV float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// A token's logits: l[i] of expert 32 i + lane, -inf where it is out of reach
// (past E, masked, or its bias masked); returns the lane's live bits
template <int NE>
MPM_DEV uint32_t route_load(const RouteArgs& a, long long t, int lane, float (&l)[NE]) {
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * 32 + lane;
    float v = -INFINITY;
    if (e < a.E) {
      if (a.bf16) v = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.logits)[t * a.ld + e] << 16);
      else v = static_cast<const float*>(a.logits)[t * a.ld + e];
      if (v > kDeadLogit && (!a.bias || a.bias[e] > kDeadLogit)) live |= 1u << i;
      v = fminf(v, kLargest);
    }
    l[i] = (live >> i & 1u) ? v : -INFINITY;
  }
  return live;
}

// scores s[i] (0 where dead) of a token from its logits, and their sum
template <int NE>
MPM_DEV float route_scores(const RouteArgs& a, const float (&l)[NE], uint32_t live, float (&s)[NE]) {
  float sum = 0.0f;
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      s[i] = (live >> i & 1u) ? __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l[i]))) : 0.0f;
      sum = __fadd_rn(sum, s[i]);
    }
    return warp_sum(sum);
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NE; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    s[i] = (live >> i & 1u) ? expf(__fsub_rn(l[i], m)) : 0.0f;
    sum = __fadd_rn(sum, s[i]);
  }
  sum = warp_sum(sum);
  const float d = sum > 0.0f ? sum : 1.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) s[i] = __fdiv_rn(s[i], d);
  return sum > 0.0f ? 1.0f : 0.0f;
}

template <int NE>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
  extern __shared__ uint8_t route_smem[];
  float* sh_load = reinterpret_cast<float*>(route_smem);             // [warps][E]
  int* sh_counts = reinterpret_cast<int*>(sh_load + kRouteWarps * a.E);   // [E]
  __shared__ int sh_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) sh_counts[e] = 0;
  if (threadIdx.x == 0) sh_n = 0;
  __syncthreads();
  float load[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) load[i] = 0.0f;
  int n = 0;
  for (long long t = (long long)blockIdx.x * kRouteWarps + warp; t < a.T;
       t += (long long)gridDim.x * kRouteWarps) {
    float l[NE], s[NE];
    const uint32_t live = route_load<NE>(a, t, lane, l);
    const float sum = route_scores<NE>(a, l, live, s);
    const bool on = !a.mask || a.mask[t] != 0;
    if (on) {
      ++n;
      const float d = sum > 0.0f ? sum : 1.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) load[i] = __fadd_rn(load[i], a.sigmoid ? __fdiv_rn(s[i], d) : s[i]);
    }
    uint32_t key[NE];                      // 0: past E or chosen; 1: dead
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 32 + lane;
      float v = l[i];
      if (a.sigmoid) v = (e < a.E && a.bias) ? __fadd_rn(s[i], a.bias[e]) : s[i];
      key[i] = e >= a.E ? 0u : ((live >> i & 1u) ? ordered_bits(v) : 1u);
    }
    float w0 = 0.0f, w1 = 0.0f, wsum = 0.0f;    // lane j: weights of choices j and 32 + j
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) best = max(best, key[i]);
      best = __reduce_max_sync(0xFFFFFFFFu, best);
      int at = 0x7FFFFFFF;
#pragma unroll
      for (int i = NE - 1; i >= 0; --i)
        if (key[i] == best) at = i * 32 + lane;
      at = __reduce_min_sync(0xFFFFFFFFu, at);
      float w = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (i * 32 + lane == at) { key[i] = 0u; w = s[i]; }
      w = __shfl_sync(0xFFFFFFFFu, w, at & 31);
      wsum = __fadd_rn(wsum, w);
      if ((j & 31) == lane) { if (j < 32) w0 = w; else w1 = w; }
      if (lane == 0) {
        a.ids[t * a.k + j] = at;
        if (on && best > 1u) atomicAdd(&sh_counts[at], 1);
      }
    }
    const float d = a.normalize && wsum > 0.0f ? wsum : 1.0f;
    if (lane < a.k) a.prob[t * a.k + lane] = on ? __fmul_rn(__fdiv_rn(w0, d), a.scale) : 0.0f;
    if (lane + 32 < a.k) a.prob[t * a.k + 32 + lane] = on ? __fmul_rn(__fdiv_rn(w1, d), a.scale) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (i * 32 + lane < a.E) sh_load[warp * a.E + i * 32 + lane] = load[i];
  if (lane == 0 && n) atomicAdd(&sh_n, n);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float v = 0.0f;
    for (int w = 0; w < kRouteWarps; ++w) v = __fadd_rn(v, sh_load[w * a.E + e]);
    a.ws_load[(long long)blockIdx.x * a.E + e] = v;
    a.ws_counts[(long long)blockIdx.x * a.E + e] = sh_counts[e];
  }
  if (threadIdx.x == 0) a.ws_n[blockIdx.x] = sh_n;
}

// the partials summed in block order: counts, mean scores, tokens, loss
__global__ void __launch_bounds__(1024) route_finish_kernel(const RouteArgs a, int parts) {
  __shared__ float sh[32];
  const int e = threadIdx.x;
  int n = 0;
  for (int i = 0; i < parts; ++i) n += a.ws_n[i];
  const float nf = (float)(n > 0 ? n : 1);
  float v = 0.0f;
  if (e < a.E) {
    float load = 0.0f;
    int c = 0;
    for (int i = 0; i < parts; ++i) {
      load = __fadd_rn(load, a.ws_load[(long long)i * a.E + e]);
      c += a.ws_counts[(long long)i * a.E + e];
    }
    load = __fdiv_rn(load, nf);
    a.load[e] = load;
    a.counts[e] = c;
    v = __fmul_rn((float)c, load);
  }
  v = warp_sum(v);
  if ((e & 31) == 0) sh[e >> 5] = v;
  __syncthreads();
  if (e == 0) {
    float s = 0.0f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s = __fadd_rn(s, sh[i]);
    *a.loss = __fdiv_rn(__fmul_rn(s, (float)a.E), __fmul_rn((float)a.k, nf));
    *a.n_tokens = n;
  }
}

// ---------------------------------------------------------------- backward
// Counts are constants; through P the loss sends dP_e = dloss E c_e / (k n^2)
// to every unmasked token's share of e.  Softmax: dl = s (ds - sum s ds).
// Sigmoid: dl = s (1 - s) ds, where a share s / S passes (dP - sum share dP) / S
// on to s.  A normalised weight q_j = s_j / W passes
// (dprob_j - sum q dprob) scale / W on to s of choice j.
template <int NE>
__global__ void __launch_bounds__(32 * kRouteWarps) route_bwd_kernel(const RouteArgs a) {
  extern __shared__ uint8_t route_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* sh = reinterpret_cast<float*>(route_smem) + warp * 2 * a.E;   // the token's s, then ds
  float* shd = sh + a.E;
  float dp[NE];                                   // dP of the lane's experts
  {
    const int n = a.in_n ? *a.in_n : 0;
    const float nf = (float)(n > 0 ? n : 1);
    const float c = (a.dloss && a.in_counts && n > 0)
                        ? __fdiv_rn(__fmul_rn(*a.dloss, (float)a.E), __fmul_rn((float)a.k, __fmul_rn(nf, nf)))
                        : 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 32 + lane;
      dp[i] = (e < a.E && a.in_counts) ? __fmul_rn(c, (float)a.in_counts[e]) : 0.0f;
    }
  }
  for (long long t = (long long)blockIdx.x * kRouteWarps + warp; t < a.T;
       t += (long long)gridDim.x * kRouteWarps) {
    const bool on = !a.mask || a.mask[t] != 0;
    float l[NE], s[NE], dl[NE];
    const uint32_t live = route_load<NE>(a, t, lane, l);
    const float sum = route_scores<NE>(a, l, live, s);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i * 32 + lane < a.E) { sh[i * 32 + lane] = s[i]; shd[i * 32 + lane] = 0.0f; }
    __syncwarp();
    if (a.dprob) {
      // lane j: choices j and 32 + j
      float w[2] = {0.0f, 0.0f}, d[2] = {0.0f, 0.0f};
      int id[2] = {-1, -1};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = c * 32 + lane;
        if (j >= a.k) continue;
        const int e = a.in_ids[t * a.k + j];
        if (e < 0 || e >= a.E) { set_status(a.status, MPM_ERR_DEVICE_BOUNDS); continue; }
        id[c] = e;
        w[c] = sh[e];
        d[c] = __fmul_rn(a.dprob[t * a.k + j], a.scale);
      }
      if (a.normalize) {
        const float W = warp_sum(__fadd_rn(w[0], w[1]));
        const float r = W > 0.0f ? __fdiv_rn(1.0f, W) : 1.0f;
        const float dot = __fmul_rn(warp_sum(__fadd_rn(__fmul_rn(w[0], d[0]), __fmul_rn(w[1], d[1]))), r);
#pragma unroll
        for (int c = 0; c < 2; ++c) d[c] = __fmul_rn(__fsub_rn(d[c], dot), r);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (id[c] >= 0) shd[id[c]] = d[c];
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) dl[i] = i * 32 + lane < a.E ? shd[i * 32 + lane] : 0.0f;
    if (a.sigmoid) {
      const float S = sum > 0.0f ? sum : 1.0f;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) dot = __fmaf_rn(s[i], dp[i], dot);
      dot = __fdiv_rn(warp_sum(dot), S);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float ds = __fadd_rn(dl[i], __fdiv_rn(__fsub_rn(dp[i], dot), S));
        // s (1 - s) = z / (1 + z)^2 with z = exp(-|l|): no cancellation at either end
        const float z = expf(-fabsf(l[i]));
        const float q = __fadd_rn(1.0f, z);
        dl[i] = __fmul_rn(__fdiv_rn(z, __fmul_rn(q, q)), ds);
      }
    } else {
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        dl[i] = __fadd_rn(dl[i], dp[i]);
        dot = __fmaf_rn(s[i], dl[i], dot);
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < NE; ++i) dl[i] = __fmul_rn(s[i], __fsub_rn(dl[i], dot));
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 32 + lane;
      if (e >= a.E) continue;
      const float v = (on && (live >> i & 1u)) ? dl[i] : 0.0f;
      if (a.bf16) static_cast<__nv_bfloat16*>(a.dlogits)[t * a.ldd + e] = __float2bfloat16_rn(v);
      else static_cast<float*>(a.dlogits)[t * a.ldd + e] = v;
    }
  }
}

// ---------------------------------------------------------------- launchers
static int route_parts(long long T) {
  const long long n = (T + kRouteWarps - 1) / kRouteWarps;
  return (int)(n < kRouteMaxParts ? n : kRouteMaxParts);
}
size_t route_ws_bytes(long long T, int E) { return (size_t)route_parts(T) * (2 * (size_t)E + 1) * 4; }

#define MPM_ROUTE_DISPATCH(E, CALL)      \
  do {                                   \
    const int ne_ = ((E) + 31) / 32;     \
    if (ne_ <= 1) { CALL(1); }           \
    else if (ne_ <= 2) { CALL(2); }      \
    else if (ne_ <= 4) { CALL(4); }      \
    else if (ne_ <= 8) { CALL(8); }      \
    else if (ne_ <= 16) { CALL(16); }    \
    else { CALL(32); }                   \
  } while (0)

cudaError_t launch_route(const RouteArgs& in, void* ws, cudaStream_t st) {
  RouteArgs a = in;
  const int parts = route_parts(a.T);
  a.ws_load = static_cast<float*>(ws);
  a.ws_counts = reinterpret_cast<int*>(a.ws_load + (size_t)parts * a.E);
  a.ws_n = a.ws_counts + (size_t)parts * a.E;
  const size_t smem = (size_t)(kRouteWarps + 1) * a.E * 4;
#define MPM_CALL(NE) route_kernel<NE><<<parts, 32 * kRouteWarps, smem, st>>>(a)
  MPM_ROUTE_DISPATCH(a.E, MPM_CALL);
#undef MPM_CALL
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  route_finish_kernel<<<1, (a.E + 31) / 32 * 32, 0, st>>>(a, parts);
  return cudaGetLastError();
}

cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t st) {
  const int parts = route_parts(a.T);
  const size_t smem = (size_t)kRouteWarps * 2 * a.E * 4;
#define MPM_CALL(NE)                                                                              \
  do {                                                                                            \
    if (smem > 48 * 1024) {                                                                       \
      cudaError_t e_ = cudaFuncSetAttribute(route_bwd_kernel<NE>,                                 \
                                            cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); \
      if (e_ != cudaSuccess) return e_;                                                           \
    }                                                                                             \
    route_bwd_kernel<NE><<<parts, 32 * kRouteWarps, smem, st>>>(a);                               \
  } while (0)
  MPM_ROUTE_DISPATCH(a.E, MPM_CALL);
#undef MPM_CALL
  return cudaGetLastError();
}

}  // namespace mpm
