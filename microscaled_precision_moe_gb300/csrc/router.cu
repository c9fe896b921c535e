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
// One warp per token, expert e in lane e % 32 (bf16: experts 2 l and 2 l + 1 of
// every 64 in lane l), so that runs of heavy experts spread over the lanes; the
// next token's logits are in flight while this one is worked on.  The choice
// compares the keys themselves, so it is exact, and ties go to the lower expert:
//   1. tau: the k-th largest of the 32 lanes' own maxima (k warp maxima; equal
//      lane maxima leave together, which can only lower tau).  At least k keys
//      are >= tau, and few more: about 10 of 256 for k = 8.
//   2. Those keys move to one lane each (their number in the lanes before by
//      ballots, the keys through shared memory), and each lane counts the keys
//      above its own, its place among the choices; only where places collide are
//      equal keys told apart by expert.
// With k > 32, more than 32 such keys (masses of ties), fewer than k lanes with an
// expert in reach or sigmoid scores that all vanish, the warp takes k maxima one after
// the other instead.
// Softmax scores use the hardware exponential (a few ulp).  A sigmoid choice
// depends on the last bit of 1 / (1 + expf(-l)), with the IEEE reciprocal, and of
// its sum with the bias: tau is found among keys by the hardware functions and
// lowered by a bound on what separates the two, and only the candidates, one a
// lane, get the exact ones (32768 x 256: 28.0 -> 25.2 us; 20000 x 400: 38.0 ->
// 29.3; 64 x 256: 5.6 -> 5.4).  Weights are of the exact scores; load and loss, sums
// over many, of the approximate ones.
// Sums over tokens go through per-block partials added in a fixed order (no
// floating-point atomics).
#include <algorithm>
#include "router.cuh"
#include "launch.cuh"
#include "packed.cuh"

namespace mpm {

constexpr int kRouteMaxParts = 152;                     // one block of up to 32 warps on each SM
constexpr int kClusterCtas = 8;
// One cluster routes up to this many tokens: no second kernel, but 8 SMs (256
// experts, sigmoid: 6.4 us at 100 tokens, 7.1 at 160; else 6.5 at 200)
constexpr long long kClusterTokens = 128;
constexpr float kDeadLogit = -3.3895313892515355e38f;   // bf16's lowest finite value
constexpr float kLargest = 3.4028234663852886e38f;
constexpr float kLog2e = 1.44269504088896341f;
// Sigmoid scores may be fp32 subnormals (logits of -88.7 to -87.3), which the
// hardware's approximations flush to 0.  Where a sum of scores is below kVanishing
// (all of its logits below -13.8) a flushed one would matter, and exact scores times
// kVanishingScale take the place of the approximate ones: the factor leaves their
// ratios as they are.  Elsewhere a flushed score is less than 2^-106 of the sum.
constexpr float kVanishing = 9.5367431640625e-7f;           // 2^-20
constexpr float kVanishingScale = 1.099511627776e12f;        // 2^40
constexpr float kLeastLogit = -88.72283f;                   // below it expf(-l) is infinite: the score is 0

// warps of a block: as many as its registers allow
constexpr int route_warps(int ne) { return ne <= 8 ? 32 : (ne <= 16 ? 16 : 8); }

// order-preserving map of a number (not NaN) to an integer above 1, and back
MPM_DEV uint32_t ordered_bits(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));      // -0 compares equal to +0
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
MPM_DEV float ordered_value(uint32_t o) {
  return __uint_as_float(o ^ ((uint32_t)((int)~o >> 31) | 0x80000000u));
}
MPM_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
MPM_DEV float warp_max(float v) { return ordered_value(__reduce_max_sync(0xFFFFFFFFu, ordered_bits(v))); }

// exp(v) for v <= 0, by the change of base 2^(v log2 e); -inf gives 0
MPM_DEV float exp_neg(float v) { return exp2_ftz(__fmul_rn(v, kLog2e)); }

// of a lane's NE (even) values
template <int NE>
MPM_DEV float lane_sum(const float (&v)[NE]) {
  uint64_t acc = f32x2(v[0], v[1]);
#pragma unroll
  for (int i = 2; i < NE; i += 2) acc = add2(acc, f32x2(v[i], v[i + 1]));
  float lo, hi;
  f32x2_split(acc, lo, hi);
  return __fadd_rn(lo, hi);
}

// the lane's i-th expert
template <bool BF16>
MPM_DEV int expert_of(int i, int lane) {
  return BF16 ? (i >> 1) * 64 + lane * 2 + (i & 1) : i * 32 + lane;
}

// A token's logits as loaded: a lane's NE values, bf16 pairs packed; -inf past E
template <int NE, bool BF16>
struct RawLogits {
  static constexpr int W = BF16 ? NE / 2 : NE;
  uint32_t w[W];
  MPM_DEV void load(const RouteArgs& a, int t, int lane) {
    if constexpr (BF16) {
      const uint16_t* p = static_cast<const uint16_t*>(a.logits) + t * a.ld + lane * 2;
      if (a.vec) {                       // even E, 4-byte aligned rows
#pragma unroll
        for (int i = 0; i < W; ++i)
          w[i] = i * 64 + lane * 2 < a.E ? *reinterpret_cast<const uint32_t*>(p + i * 64) : 0xFF80FF80u;
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int e = i * 64 + lane * 2;
          const uint32_t lo = e < a.E ? p[i * 64] : 0xFF80u;
          const uint32_t hi = e + 1 < a.E ? p[i * 64 + 1] : 0xFF80u;
          w[i] = lo | (hi << 16);
        }
      }
    } else {
      const uint32_t* p = static_cast<const uint32_t*>(a.logits) + t * a.ld + lane;
      if (a.vec) {                       // E = 32 NE
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = p[i * 32];
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = i * 32 + lane < a.E ? p[i * 32] : 0xFF800000u;
      }
    }
  }
  MPM_DEV float value(int i) const {
    if constexpr (BF16) return (i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
    else return __uint_as_float(w[i]);
  }
};

// Logits with -inf for what is out of reach; dead_bias: the lane's experts
// whose bias puts them there
template <int NE, bool BF16>
MPM_DEV void route_logits(const RawLogits<NE, BF16>& raw, uint32_t dead_bias, float (&l)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const float v = raw.value(i);
    l[i] = (v > kDeadLogit && !(dead_bias >> i & 1u)) ? fminf(v, kLargest) : -INFINITY;
  }
}

template <int NE, bool BF16>
MPM_DEV uint32_t route_bias(const RouteArgs& a, int lane, float (&bias)[NE]) {
  uint32_t dead = 0;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = expert_of<BF16>(i, lane);
    bias[i] = (a.bias && e < a.E) ? a.bias[e] : 0.0f;
    if (!(bias[i] > kDeadLogit)) dead |= 1u << i;
  }
  return dead;
}

// ---------------------------------------------------------------- forward
// k maxima one after the other, lowest expert first among equals, those out of
// reach last: ids, weights and counts of a token
template <int NE, bool BF16>
MPM_DEV void route_one_by_one(const RouteArgs& a, int t, int lane, const float (&key)[NE],
                              const float (&s)[NE], float unit, bool on, int* sh_counts) {
  uint32_t taken = 0;
  float w0 = 0.0f, w1 = 0.0f, d = 0.0f;                 // lane j: weights of choices j and 32 + j
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
    int at = 0x7FFFFFFF, slot = 0;
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = expert_of<BF16>(i, lane);
      uint32_t o = key[i] > -INFINITY ? ordered_bits(key[i]) : 1u;
      if (e >= a.E || (taken >> i & 1u)) o = 0u;
      if (o > best) { best = o; at = e; slot = i; w = s[i]; }
    }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const int e = __reduce_min_sync(0xFFFFFFFFu, best == top ? at : 0x7FFFFFFF);
    if (e == at) taken |= 1u << slot;
    w = __shfl_sync(0xFFFFFFFFu, w, __ffs(__ballot_sync(0xFFFFFFFFu, e == at)) - 1);
    d = __fadd_rn(d, w);
    if ((j & 31) == lane) { if (j < 32) w0 = w; else w1 = w; }
    if (lane == 0) {
      a.ids[t * a.k + j] = e;
      if (on && top > 1u) atomicAdd(&sh_counts[e], 1);
    }
  }
  float f = unit;
  if (a.normalize) {
    if (d < kVanishing) {                               // sigmoid scores only, or none in reach
      w0 = __fmul_rn(w0, kVanishingScale);
      w1 = __fmul_rn(w1, kVanishingScale);
      d = __fmul_rn(d, kVanishingScale);
    }
    f = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
  }
  if (lane < a.k) a.prob[t * a.k + lane] = on ? __fmul_rn(__fmul_rn(w0, f), a.scale) : 0.0f;
  if (lane + 32 < a.k) a.prob[t * a.k + 32 + lane] = on ? __fmul_rn(__fmul_rn(w1, f), a.scale) : 0.0f;
}

// a warp's shared memory in the token loop: the candidates' keys and experts
struct __align__(16) RouteWarp {
  float key[32];
  int expert[32];
};

// The lane's keys >= least, and their experts, to the places from `to` (shared
// memory) on.  Two predicated stores and an addition a key: as a conditional the
// compiler spent twice as many instructions.
template <int NE, bool BF16>
MPM_DEV void put_candidates(const float (&key)[NE], float least, int lane, uint32_t to) {
#pragma unroll
  for (int i = 0; i < NE; ++i)
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ge.f32 p, %1, %2;\n\t"
                 "@p st.shared.f32 [%0], %1;\n\t"
                 "@p st.shared.u32 [%0 + 128], %3;\n\t"
                 "@p add.u32 %0, %0, 4;\n\t}"
                 : "+r"(to) : "f"(key[i]), "f"(least), "r"(expert_of<BF16>(i, lane)) : "memory");
}

// what the choice compares: the logits, or sigmoid scores with their bias
template <bool SIG, int NE>
MPM_DEV float (&route_keys(float (&l)[NE], float (&sig_key)[SIG ? NE : 1]))[NE] {
  if constexpr (SIG) return sig_key;
  else return l;
}

MPM_DEV float sigmoid_exact(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }
// 1 / (1 + 2^(-l log2 e)) by the hardware functions.  With u = 2^-24 and z = e^-l:
// z is off by (1.5 |l| + 4) u of itself and s by (1 - s) of that and 3 u; since
// s (1 - s) |l| < 0.23 it is within 5 u of the true s absolutely, and within
// (1.5 |l| + 7) u < 140 u of it relatively where z is below 2^126; the exact form
// is within 3 u and 6 u.
MPM_DEV float sigmoid_fast(float l) { return rcp_ftz(__fadd_rn(1.0f, exp2_ftz(__fmul_rn(l, -kLog2e)))); }
// What to lower tau by so that every exact key among the k largest is a
// candidate: twice the most that the two keys of an expert differ by, and more.
// Without a bias relatively (twice 146 u, 1.7e-5), so that small scores do not all
// become candidates, with one 16 u and the rounding of two sums, 4 u |key|.
MPM_DEV float sigmoid_margin(float tau, bool biased) {
  return biased ? __fmaf_rn(fabsf(tau), 1e-6f, 2e-6f) : fminf(2e-6f, __fmul_rn(tau, 5e-5f));
}

// One token: ids and weights to global memory, counts to sh_counts, shares
// added to load.  raw: its logits; replaced by those of token `next`.
template <int NE, bool SIG, bool BF16>
MPM_DEV void route_token(const RouteArgs& a, int t, int next, int lane, RawLogits<NE, BF16>& raw,
                         bool on, uint32_t dead_bias, const float (&bias)[NE], float (&load)[NE],
                         int* sh_counts, RouteWarp& sh) {
  float l[NE], s[NE], sig_key[SIG ? NE : 1];
  float top = -INFINITY, sum = 0.0f;
  if constexpr (SIG) {
    route_logits<NE, BF16>(raw, dead_bias, l);
  } else {
    // What is out of reach shows later: NaN in the sum, the rest in tau and the maximum
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      l[i] = raw.value(i);
      top = fmaxf(top, l[i]);            // the number, where one is NaN
    }
  }
  if (next < (int)a.T) raw.load(a, next, lane);
  if constexpr (SIG) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {       // (by pairs: 26.4 against 24.7 us at 32768 x 256)
      s[i] = sigmoid_fast(l[i]);         // l = -inf: 2^inf, and the score is 0
      sig_key[i] = l[i] > -INFINITY ? __fadd_rn(s[i], bias[i]) : -INFINITY;
      top = fmaxf(top, sig_key[i]);
    }
  }
  float (&key)[NE] = route_keys<SIG, NE>(l, sig_key);
  uint32_t o = ordered_bits(top);
  uint32_t tau = __reduce_max_sync(0xFFFFFFFFu, o);
  float m = ordered_value(tau);
  if (a.k <= 8) {                        // without branches: all of eight rounds, the k-th kept
    uint32_t v = tau;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      if (o == v) o = 0;
      v = __reduce_max_sync(0xFFFFFFFFu, o);
      if (j < a.k) tau = v;
    }
  } else {
    for (int j = 1; j < a.k; ++j) {
      if (o == tau) o = 0;
      tau = __reduce_max_sync(0xFFFFFFFFu, o);
    }
  }
  const float least = ordered_value(tau);               // tau = 0 (lanes ran out): NaN
  bool quick = least > kDeadLogit && a.k <= 32;
  float cut = least;
  if constexpr (SIG) {
    cut = __fsub_rn(least, sigmoid_margin(least, a.bias != nullptr));
    // not where scores may have been flushed to 0, nor for an infinite bias (cut: NaN)
    quick = quick && (a.bias || least > 1e-30f) && cut > -INFINITY;
  }
  float m2 = 0.0f;
  if constexpr (!SIG) {
    if (quick && fabsf(m) < 32768.0f) {
      // exp(l - m) as 2^(l log2 e - m log2 e), the product exact within the
      // FMA: the rounding of m log2 e is one factor, below 1.003, of all s
      m2 = __fmul_rn(m, kLog2e);
      const uint64_t scale2 = f32x2(kLog2e, kLog2e), from2 = f32x2(-m2, -m2);
#pragma unroll
      for (int i = 0; i < NE; i += 2) {
        f32x2_split(fma2(f32x2(l[i], l[i + 1]), scale2, from2), s[i], s[i + 1]);
        s[i] = exp2_ftz(s[i]);
        s[i + 1] = exp2_ftz(s[i + 1]);
      }
      sum = warp_sum(lane_sum(s));
      quick = sum == sum;
    } else {
      quick = false;
    }
    if (!quick) {
      RawLogits<NE, BF16> again;
      again.load(a, t, lane);
      route_logits<NE, BF16>(again, 0u, l);
      m = fminf(fmaxf(m, -kLargest), kLargest);         // none in reach: exp(-inf) = 0
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = exp_neg(__fsub_rn(l[i], m));
      sum = warp_sum(lane_sum(s));
    }
  } else {
    sum = warp_sum(lane_sum(s));
    quick = quick && sum >= kVanishing;  // else the shares are taken below
  }
  const float share = on && sum >= kVanishing ? rcp_ftz(sum) : 0.0f;      // (softmax: 0, or 1 and more)
  const uint64_t share2 = f32x2(share, share);
#pragma unroll
  for (int i = 0; i < NE; i += 2)
    f32x2_split(fma2(f32x2(s[i], s[i + 1]), share2, f32x2(load[i], load[i + 1])), load[i], load[i + 1]);
  // a weight before normalisation is s times this
  const float unit = SIG ? 1.0f : share;
  if (quick) {
    const uint32_t below_lane = (1u << lane) - 1u;
    int c = 0;                           // the lane's candidates
#pragma unroll
    for (int i = 0; i < NE; ++i) c += key[i] >= cut ? 1 : 0;
    // the sum of c over the lanes before, bit by bit: seldom more than two
    int at = 0, n = 0;
    auto add_bit = [&](int bit) {
      const uint32_t b = __ballot_sync(0xFFFFFFFFu, c >> bit & 1);
      at += __popc(b & below_lane) << bit;
      n += __popc(b) << bit;
    };
    add_bit(0);
    add_bit(1);
    for (int bit = 2; __any_sync(0xFFFFFFFFu, c >> bit); ++bit) add_bit(bit);
    if (n <= 32) {
      __syncwarp();                      // the previous token's candidates have been read
      put_candidates<NE, BF16>(key, cut, lane, smem_u32(&sh.key[at]));
      if (lane >= n) sh.key[lane] = -INFINITY;
      __syncwarp();
      // lane j has candidate j, in no particular order; of 16 or fewer, lane j + 16
      // has it too and looks at the other half of them
      const bool few = n <= 16;
      const int seat = few ? lane & 15 : lane;
      float own = sh.key[seat], w = 0.0f;
      const int e = seat < n ? sh.expert[seat] : 0;
      if constexpr (SIG) {
        float v, b = 0.0f;
        if constexpr (BF16) v = bf16lo(static_cast<const uint16_t*>(a.logits)[t * a.ld + e]);
        else v = static_cast<const float*>(a.logits)[t * a.ld + e];
        if (a.bias) b = a.bias[e];
        w = sigmoid_exact(fminf(v, kLargest));
        if (seat < n) own = __fadd_rn(w, b);
        __syncwarp();
        sh.key[seat] = own;              // of two lanes with one seat, the same
        __syncwarp();
      }
      int place = 0;
      auto count = [&](int j) {
        const float4 q = *reinterpret_cast<const float4*>(&sh.key[j]);
        place += (q.x > own ? 1 : 0) + (q.y > own ? 1 : 0) + (q.z > own ? 1 : 0) + (q.w > own ? 1 : 0);
      };
      if (few) {
        const int j0 = lane >> 4 << 3;
#pragma unroll
        for (int j = 0; j < 8; j += 4) count(j0 + j);
        place += __shfl_xor_sync(0xFFFFFFFFu, place, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 32; j += 4) count(j);
      }
      bool chosen = lane < n && place < a.k;
      // Equal keys share a place: then k lanes do not hold the k places.  Where k
      // lanes are chosen, their places' powers of two add up to 2^k - 1 only if
      // no two are the same (k <= 16: with their number in the bits above).
      bool apart;
      if (a.k <= 16) {
        const uint32_t held = __reduce_add_sync(0xFFFFFFFFu, chosen ? (1u << place) + (1u << 24) : 0u);
        apart = held == (1u << a.k) - 1u + ((uint32_t)a.k << 24);
      } else {
        const uint32_t held = __reduce_or_sync(0xFFFFFFFFu, chosen ? 1u << place : 0u);
        apart = __popc(held) == a.k && __popc(__ballot_sync(0xFFFFFFFFu, chosen)) == a.k;
      }
      if (!apart) {
        for (int j = 0; j < n; ++j)
          place += sh.key[j] == own && sh.expert[j] < e ? 1 : 0;
        chosen = lane < n && place < a.k;
      }
      if constexpr (SIG) w = chosen ? w : 0.0f;
      else w = chosen ? exp2_ftz(__fmaf_rn(own, kLog2e, -m2)) : 0.0f;
      float f = unit;
      if (a.normalize) {
        float d = warp_sum(w);
        if (SIG && d < kVanishing) {
          w = __fmul_rn(w, kVanishingScale);
          d = __fmul_rn(d, kVanishingScale);
        }
        f = d > 0.0f ? rcp_ftz(d) : 0.0f;
      }
      if (chosen) {
        const int to = t * a.k + place;
        a.ids[to] = e;
        a.prob[to] = on ? __fmul_rn(__fmul_rn(w, f), a.scale) : 0.0f;
        if (on) atomicAdd(&sh_counts[e], 1);
      }
      return;
    }
  }
  RawLogits<NE, BF16> again;
  again.load(a, t, lane);
  route_logits<NE, BF16>(again, dead_bias, l);
  if constexpr (SIG) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      s[i] = sigmoid_exact(l[i]);
      sig_key[i] = l[i] > -INFINITY ? __fadd_rn(s[i], bias[i]) : -INFINITY;
    }
    if (on && sum < kVanishing) {
      sum = __fmul_rn(warp_sum(lane_sum(s)), kVanishingScale);
      const float f = sum > 0.0f ? rcp_ftz(sum) : 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) load[i] = __fmaf_rn(__fmul_rn(s[i], kVanishingScale), f, load[i]);
    }
  }
  route_one_by_one<NE, BF16>(a, t, lane, key, s, unit, on, sh_counts);
}

// totals of expert e over all tokens -> counts and load; returns its part of the loss
MPM_DEV float route_expert_totals(const RouteArgs& a, int e, float load, int c, float n) {
  load = __fdiv_rn(load, n);
  a.load[e] = load;
  a.counts[e] = c;
  return __fmul_rn((float)c, load);
}
MPM_DEV void route_totals(const RouteArgs& a, float loss, int n) {
  const float nf = (float)(n > 0 ? n : 1);
  *a.loss = __fdiv_rn(__fmul_rn(loss, (float)a.E), __fmul_rn((float)a.k, nf));
  *a.n_tokens = n;
}

MPM_DEV uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}

// Bound by its instructions, about 420 a token at E = 256, k = 8 (80 % of the
// issue slots; DRAM at a quarter): 32768 tokens take 18.5 us, 3.7 of them in the
// sum over blocks below, where reading the logits would take 5.  Slopes: 1.9 us
// per 4864 tokens, 1.5 at E = 64, k = 4, the same for k = 1: mostly a token's
// fixed steps.  A warp per token and k arg-max rounds over all keys took 110 us.
//
// Shared memory: the block's loads [E] and counts [E], then a region that
// holds the warps' candidates during the token loop and their lanes' loads
// [warps][E] after it
template <int NE, bool SIG, bool BF16>
__global__ void __launch_bounds__(32 * route_warps(NE)) route_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) uint8_t route_smem[];
  float* sh_load = reinterpret_cast<float*>(route_smem);
  int* sh_counts = reinterpret_cast<int*>(sh_load + a.E);
  uint8_t* region = route_smem + (size_t)(2 * a.E + 3) / 4 * 16;
  float* sh_part = reinterpret_cast<float*>(region);
  __shared__ int sh_n[32];
  __shared__ float sh_loss;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = blockDim.x >> 5;
  RouteWarp& sh = reinterpret_cast<RouteWarp*>(region)[warp];
  const int step = gridDim.x * W, T = (int)a.T;         // T k <= 2^30
  int t = blockIdx.x * W + warp;
  RawLogits<NE, BF16> raw;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) sh_counts[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  if (t < T) raw.load(a, t, lane);
  float load[NE], bias[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) load[i] = 0.0f;
  const uint32_t dead_bias = SIG ? route_bias<NE, BF16>(a, lane, bias) : 0u;
  __syncthreads();
  int n = 0;
  while (t < T) {
    const bool on = !a.mask || a.mask[t] != 0;
    const int next = t + step;
    route_token<NE, SIG, BF16>(a, t, next, lane, raw, on, dead_bias, bias, load, sh_counts, sh);
    n += on ? 1 : 0;
    t = next;
  }
  if (lane == 0) sh_n[warp] = n;
  __syncthreads();                       // the region is free
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = expert_of<BF16>(i, lane);
    if (e < a.E) sh_part[warp * a.E + e] = load[i];
  }
  __syncthreads();
  n = __reduce_add_sync(0xFFFFFFFFu, lane < W ? sh_n[lane] : 0);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float v = 0.0f;
#pragma unroll 8
    for (int w = 0; w < W; ++w) v = __fadd_rn(v, sh_part[w * a.E + e]);
    if (a.cluster) {
      sh_load[e] = v;
    } else {
      a.ws_load[(long long)blockIdx.x * a.E + e] = v;
      a.ws_counts[(long long)blockIdx.x * a.E + e] = sh_counts[e];
    }
  }
  if (!a.cluster) {
    if (threadIdx.x == 0) a.ws_n[blockIdx.x] = n;
    return;
  }
  // one cluster of 8 blocks holds every token: block r adds up the experts e = r mod 8
  __syncthreads();                       // sh_n read by every thread
  if (threadIdx.x == 0) sh_n[0] = n;
  const uint32_t rank = cluster_ctarank();
  cluster_sync();
  int nc[kClusterCtas];
#pragma unroll
  for (int c = 0; c < kClusterCtas; ++c) nc[c] = (int)ld_cluster_u32(&sh_n[0], c);
  float loss = 0.0f;
  for (int e = threadIdx.x * kClusterCtas + rank; e < a.E; e += blockDim.x * kClusterCtas) {
    uint32_t lc[kClusterCtas], cc[kClusterCtas];
#pragma unroll
    for (int c = 0; c < kClusterCtas; ++c) {
      lc[c] = ld_cluster_u32(&sh_load[e], c);
      cc[c] = ld_cluster_u32(&sh_counts[e], c);
    }
    n = 0;
    float v = 0.0f;
    int k = 0;
#pragma unroll
    for (int c = 0; c < kClusterCtas; ++c) {
      n += nc[c];
      v = __fadd_rn(v, __uint_as_float(lc[c]));
      k += (int)cc[c];
    }
    loss = __fadd_rn(loss, route_expert_totals(a, e, v, k, (float)(n > 0 ? n : 1)));
  }
  loss = warp_sum(loss);
  if (lane == 0) sh_part[warp] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < W; ++w) loss = __fadd_rn(loss, sh_part[w]);
    sh_loss = loss;
  }
  cluster_sync();
  if (rank == 0 && warp == 0) {
    n = 0;
#pragma unroll
    for (int c = 0; c < kClusterCtas; ++c) n += nc[c];
    loss = warp_sum(lane < kClusterCtas ? __uint_as_float(ld_cluster_u32(&sh_loss, lane)) : 0.0f);
    if (lane == 0) route_totals(a, loss, n);
  }
  cluster_sync();                        // no block leaves while its shared memory is read
}

// The blocks' partials summed: one cluster of 8 blocks, each taking every 8th
// group of 32 experts, warp w the parts w, w + 32, ... of them.  Latency only
// (300 KB from L2): 3.7 us behind the kernel before; one block took 2.8 more.
__global__ void __launch_bounds__(1024) route_finish_kernel(const RouteArgs a, int parts) {
  __shared__ float sh_l[32][33];
  __shared__ int sh_c[32][33];
  __shared__ int sh_n[32];
  __shared__ float sh_loss;
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  int n = 0;
  const int my_n = (int)threadIdx.x < parts ? a.ws_n[threadIdx.x] : 0;     // parts <= 152
  float loss = 0.0f;
  for (int e0 = (int)rank * 32; e0 < a.E; e0 += kClusterCtas * 32) {
    const int e = e0 + lane;
    float v = 0.0f;
    int c = 0;
    if (e < a.E) {
#pragma unroll 5
      for (int i = warp; i < parts; i += 32) {
        v = __fadd_rn(v, a.ws_load[(long long)i * a.E + e]);
        c += a.ws_counts[(long long)i * a.E + e];
      }
    }
    n = __reduce_add_sync(0xFFFFFFFFu, my_n);             // after the loads above are out
    if (lane == 0) sh_n[warp] = n;
    sh_l[warp][lane] = v;
    sh_c[warp][lane] = c;
    __syncthreads();
    // warp w: the 32 partial sums of expert e0 + w
    v = warp_sum(sh_l[lane][warp]);
    c = __reduce_add_sync(0xFFFFFFFFu, sh_c[lane][warp]);
    n = __reduce_add_sync(0xFFFFFFFFu, sh_n[lane]);
    if (lane == 0 && e0 + warp < a.E)
      loss = __fadd_rn(loss, route_expert_totals(a, e0 + warp, v, c, (float)(n > 0 ? n : 1)));
    __syncthreads();
  }
  if (lane == 0) sh_l[0][warp] = loss;
  __syncthreads();
  if (warp == 0) {
    loss = warp_sum(sh_l[0][lane]);
    n = __reduce_add_sync(0xFFFFFFFFu, sh_n[lane]);
    if (lane == 0) sh_loss = loss;
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    for (uint32_t c = 1; c < kClusterCtas; ++c)
      loss = __fadd_rn(loss, __uint_as_float(ld_cluster_u32(&sh_loss, c)));
    route_totals(a, loss, n);
  }
  cluster_sync();
}

// ---------------------------------------------------------------- backward
// Counts are constants; through P the loss sends dP_e = dloss E c_e / (k n^2)
// to every unmasked token's share of e.  Softmax: dl = s (ds - sum s ds).
// Sigmoid: dl = s (1 - s) ds, where a share s / S passes (dP - sum share dP) / S
// on to s.  A normalised weight q_j = s_j / W passes
// (dprob_j - sum q dprob) scale / W on to s of choice j.
// Scores: softmax numerators over a common sum; sigmoid with z = exp(-|l|) as
// 1 / (1 + z) or z / (1 + z), and s (1 - s) = z / (1 + z)^2, without
// cancellation at either end.  The choices' scores are recomputed from their
// logits (one lane each), and their ds join the others through shared memory.
// The sigmoid's dl is a product of s, as small as fp32 goes, and 1 / S or 1 / W, as
// large: s and s (1 - s) are held times 2^40, which keeps each factor in fp32's range
// (for gradients up to 10^12 where the sums are smallest, down to 10^-33 where they
// are not) and cancels in s / S and s / W.  A branch for vanishing sums instead: 23.7
// against 24.6 us at 32768 x 256, 21.5 and 21.2 with bf16 logits.  exp(-|l|), which
// may be a subnormal, is the square of the hardware's exp(-|l| / 2), which is not.
MPM_DEV float sigmoid_parts(float l, float& slope) {
  const float e = exp2_ftz(__fmul_rn(-fabsf(l), 0.5f * kLog2e));
  const float z = l >= kLeastLogit ? __fmul_rn(e, e) : 0.0f;
  const float q = rcp_ftz(__fadd_rn(1.0f, z)), qs = __fmul_rn(q, kVanishingScale), zq = __fmul_rn(z, qs);
  slope = __fmul_rn(zq, q);
  return l >= 0.0f ? qs : zq;
}

// A warp per token, the next token's logits in flight.  8191 tokens of 128 bf16
// experts take 4.9 us (reading and writing the logits: 0.7): the chain of five warp
// sums and two passes through shared memory of a warp's one or two tokens, and
// the launch.  Without the next token in flight, scores through shared memory: 9.3 us.
constexpr int kBwdWarps = 8;
// Blocks an SM, which is also the grid: with more blocks than are resident some
// warps have a token more than the others (32768 x 256: 23.7 us with 6 an SM,
// 19.9 with the 4 that fit; 8191 x 128: 5.5 with 5 resident of 6, 4.9 with all 6)
constexpr int bwd_blocks(int ne, bool sig) {
  return ne <= 2 ? 8 : ne <= 4 ? (sig ? 5 : 6) : ne <= 8 ? 4 : ne <= 16 ? (sig ? 2 : 3) : 1;
}

template <int NE, bool SIG, bool BF16>
__global__ void __launch_bounds__(32 * kBwdWarps, bwd_blocks(NE, SIG)) route_bwd_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) uint8_t route_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* shd = reinterpret_cast<float*>(route_smem) + warp * (32 * NE);      // the token's ds
  const int step = gridDim.x * kBwdWarps, T = (int)a.T;      // T k <= 2^30
  int t = blockIdx.x * kBwdWarps + warp;
  RawLogits<NE, BF16> raw;
  pdl_wait();
  pdl_launch_dependents();
  if (t < T) raw.load(a, t, lane);
  float dp[NE], bias[NE];                         // dP of the lane's experts
  const uint32_t dead_bias = SIG ? route_bias<NE, BF16>(a, lane, bias) : 0u;
  {
    const int n = a.in_n ? *a.in_n : 0;
    const float nf = (float)(n > 0 ? n : 1);
    const float c = (a.dloss && n > 0)
                        ? __fdiv_rn(__fmul_rn(*a.dloss, (float)a.E), __fmul_rn((float)a.k, __fmul_rn(nf, nf)))
                        : 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = expert_of<BF16>(i, lane);
      dp[i] = (e < a.E && a.dloss) ? __fmul_rn(c, (float)a.in_counts[e]) : 0.0f;
    }
  }
  while (t < T) {
    const bool on = !a.mask || a.mask[t] != 0;
    // the choices' logits and gradients: lane j has choices j and 32 + j
    float cl[2] = {-INFINITY, -INFINITY}, d[2] = {0.0f, 0.0f};
    int id[2] = {-1, -1};
    if (a.dprob) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = c * 32 + lane;
        if (j >= a.k) continue;
        const int e = a.in_ids[t * a.k + j];
        if (e < 0 || e >= a.E) { set_status(a.status, MPM_ERR_DEVICE_BOUNDS); continue; }
        id[c] = e;
        float v;
        if constexpr (BF16) v = bf16lo(static_cast<const uint16_t*>(a.logits)[t * a.ld + e]);
        else v = static_cast<const float*>(a.logits)[t * a.ld + e];
        if (v > kDeadLogit && (!SIG || !a.bias || a.bias[e] > kDeadLogit)) cl[c] = fminf(v, kLargest);
        d[c] = __fmul_rn(a.dprob[t * a.k + j], a.scale);
      }
    }
    float l[NE], s[NE], dl[NE];
    route_logits<NE, BF16>(raw, dead_bias, l);
    const int next = t + step;
    if (next < T) raw.load(a, next, lane);
    float sum = 0.0f, m = l[0];
    if constexpr (SIG) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        s[i] = sigmoid_parts(l[i], dl[i]);        // dl: the slope s (1 - s), for now
        sum = __fadd_rn(sum, s[i]);
      }
    } else {
#pragma unroll
      for (int i = 1; i < NE; ++i) m = fmaxf(m, l[i]);
      m = fmaxf(warp_max(m), -kLargest);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        s[i] = exp_neg(__fsub_rn(l[i], m));
        sum = __fadd_rn(sum, s[i]);
      }
    }
    sum = warp_sum(sum);
    const float r = sum > 0.0f ? rcp_ftz(sum) : 0.0f;                // shares: s r
    float ds[NE];
    if (a.dprob) {
      if (a.normalize) {
        float w[2], slope;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          w[c] = SIG ? sigmoid_parts(cl[c], slope) : __fmul_rn(exp_neg(__fsub_rn(cl[c], m)), r);
        const float wsum = warp_sum(__fadd_rn(w[0], w[1]));
        const float rw = wsum > 0.0f ? __fdiv_rn(1.0f, wsum) : 1.0f;
        const float dot = warp_sum(__fmaf_rn(__fmul_rn(w[0], rw), d[0], __fmul_rn(__fmul_rn(w[1], rw), d[1])));
#pragma unroll
        for (int c = 0; c < 2; ++c) d[c] = __fmul_rn(__fsub_rn(d[c], dot), rw);
      } else if (SIG) {
#pragma unroll
        for (int c = 0; c < 2; ++c) d[c] = __fmul_rn(d[c], 1.0f / kVanishingScale);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NE; ++i) shd[i * 32 + lane] = 0.0f;
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (id[c] >= 0) shd[id[c]] = d[c];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NE; ++i) ds[i] = shd[expert_of<BF16>(i, lane)];
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) ds[i] = 0.0f;
    }
    float dot = 0.0f;
    if constexpr (SIG) {
#pragma unroll
      for (int i = 0; i < NE; ++i) dot = __fmaf_rn(s[i], dp[i], dot);
      dot = __fmul_rn(warp_sum(dot), r);
#pragma unroll
      for (int i = 0; i < NE; ++i) dl[i] = __fmul_rn(dl[i], __fmaf_rn(__fsub_rn(dp[i], dot), r, ds[i]));
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        s[i] = __fmul_rn(s[i], r);
        ds[i] = __fadd_rn(ds[i], dp[i]);
        dot = __fmaf_rn(s[i], ds[i], dot);
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < NE; ++i) dl[i] = __fmul_rn(s[i], __fsub_rn(ds[i], dot));
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) dl[i] = (on && l[i] > -INFINITY) ? dl[i] : 0.0f;
    if (a.out_bf16) {
      __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.dlogits) + t * a.ldd;
#pragma unroll
      for (int i = 0; i < NE; i += BF16 ? 2 : 1) {
        const int e = expert_of<BF16>(i, lane);
        if (BF16 && a.vec_out) {               // even E, 4-byte aligned rows
          if (e < a.E) *reinterpret_cast<__nv_bfloat162*>(p + e) = __floats2bfloat162_rn(dl[i], dl[(i + 1) % NE]);
        } else {
          if (e < a.E) p[e] = __float2bfloat16_rn(dl[i]);
          if (BF16 && e + 1 < a.E) p[e + 1] = __float2bfloat16_rn(dl[(i + 1) % NE]);
        }
      }
    } else {
      float* p = static_cast<float*>(a.dlogits) + t * a.ldd;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (expert_of<BF16>(i, lane) < a.E) p[expert_of<BF16>(i, lane)] = dl[i];
    }
    t = next;
  }
}

// ---------------------------------------------------------------- launchers
static int route_ne(int E) {
  int ne = 2;
  while (ne * 32 < E) ne *= 2;
  return ne;
}
// Warps of a block outside the cluster: as many as its registers allow, but few
// tokens are spread over the SMs, down to 8 a block (512 tokens of 256 experts,
// sigmoid: 7.9 us by 32 warps, 6.7 by 8, 7.2 by 4 and twice the partials)
static int route_block_warps(long long T, int E) {
  const int most = route_warps(route_ne(E));
  const long long w = (T + kRouteMaxParts - 1) / kRouteMaxParts;
  return (int)std::min<long long>(most, std::max<long long>(w, 8));
}
static int route_parts(long long T, int E) {
  const int w = route_block_warps(T, E);
  const long long n = (T + w - 1) / w;
  return (int)(n < kRouteMaxParts ? n : kRouteMaxParts);
}
size_t route_ws_bytes(long long T, int E) {
  return T <= kClusterTokens ? 0 : (size_t)route_parts(T, E) * (2 * (size_t)E + 1) * 4;
}
// bf16: whether rows can be read in pairs; fp32: whether every lane's slot is full
static bool route_vec(const void* p, long long ld, int bf16, int E) {
  if (!bf16) return E == 32 * route_ne(E);
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0 && E % 2 == 0;
}

template <int NE, bool SIG, bool BF16>
static cudaError_t route_forward(RouteArgs a, cudaStream_t st) {
  const bool small = a.T <= kClusterTokens;
  int W = small ? route_warps(NE) : route_block_warps(a.T, a.E);
  if (small && a.T < (long long)kClusterCtas * W) W = (int)std::max<long long>((a.T + kClusterCtas - 1) / kClusterCtas, 4);   // four for the sums
  const size_t warp_bytes = std::max(sizeof(RouteWarp), (size_t)a.E * 4);
  const size_t smem = (size_t)(2 * a.E + 3) / 4 * 16 + W * warp_bytes;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kClusterCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  if (small) {
    cfg.gridDim = dim3(kClusterCtas);
    cfg.numAttrs = 2;
    a.cluster = 1;
    return cudaLaunchKernelEx(&cfg, route_kernel<NE, SIG, BF16>, a);
  }
  const int parts = route_parts(a.T, a.E);
  cfg.gridDim = dim3((unsigned)parts);
  cfg.numAttrs = 1;
  cudaError_t err = cudaLaunchKernelEx(&cfg, route_kernel<NE, SIG, BF16>, a);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3(kClusterCtas);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, route_finish_kernel, a, parts);
}

template <int NE, bool SIG, bool BF16>
static cudaError_t route_backward(RouteArgs a, cudaStream_t st) {
  const long long n = (a.T + kBwdWarps - 1) / kBwdWarps, most = 152 * bwd_blocks(NE, SIG);
  return launch_serial(route_bwd_kernel<NE, SIG, BF16>, dim3((unsigned)(n < most ? n : most)),
                       dim3(32 * kBwdWarps), (size_t)kBwdWarps * 32 * NE * 4, st, a);
}

#define MPM_ROUTE_NE(CALL, NE)                                               \
  return a.sigmoid ? (a.bf16 ? CALL<NE, true, true>(a, st) : CALL<NE, true, false>(a, st))     \
                   : (a.bf16 ? CALL<NE, false, true>(a, st) : CALL<NE, false, false>(a, st))
#define MPM_ROUTE_DISPATCH(CALL)        \
  switch (route_ne(a.E)) {              \
    case 2: MPM_ROUTE_NE(CALL, 2);      \
    case 4: MPM_ROUTE_NE(CALL, 4);      \
    case 8: MPM_ROUTE_NE(CALL, 8);      \
    case 16: MPM_ROUTE_NE(CALL, 16);    \
    default: MPM_ROUTE_NE(CALL, 32);    \
  }

cudaError_t launch_route(const RouteArgs& in, void* ws, cudaStream_t st) {
  RouteArgs a = in;
  const size_t parts = (size_t)route_parts(a.T, a.E);
  a.ws_load = static_cast<float*>(ws);
  a.ws_counts = reinterpret_cast<int*>(a.ws_load + parts * a.E);
  a.ws_n = a.ws_counts + parts * a.E;
  a.vec = route_vec(a.logits, a.ld, a.bf16, a.E);
  MPM_ROUTE_DISPATCH(route_forward)
}

cudaError_t launch_route_backward(const RouteArgs& in, cudaStream_t st) {
  RouteArgs a = in;
  a.vec = route_vec(a.logits, a.ld, a.bf16, a.E);
  a.vec_out = route_vec(a.dlogits, a.ldd, 1, a.E);
  MPM_ROUTE_DISPATCH(route_backward)
}

}  // namespace mpm
