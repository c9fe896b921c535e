// Device helpers of the MXFP8 encoding, shared by the quantisers (quant.cu)
// and the norm's 8-bit output (norm.cu), so that both give the same bytes.
#pragma once
#include "common.cuh"

namespace mpm {

// {s, s} as the operand of a packed f32x2 multiply
MPM_DEV uint64_t f32x2_splat(float s) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %1};" : "=l"(v) : "f"(s));
  return v;
}
// the bf16 pair in w (low half first) times a power of two, then packed to
// E4M3 (RN, satfinite, low byte first).  Both lanes go through one packed
// f32x2 multiply: per lane the same IEEE product as a scalar multiply (exact
// here), so the codes are those of the scalar path.
MPM_DEV uint32_t e4m3x2_scaled(uint32_t w, uint64_t sc2) {
  uint64_t v, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(bf16lo(w)), "f"(bf16hi(w)));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(v), "l"(sc2));
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(out) : "f"(lo), "f"(hi));
  return out;
}

// Scale exponent e of a block whose |max| has the fp32 bit pattern `bits`:
// the smallest e with a <= 448 * 2^e, clamped to [-127, 127].  For
// a = 1.f * 2^p:  e = p - 8 + [1.f > 1.75].  Zero and subnormal a clamp to -127.
MPM_DEV int mx_exponent(uint32_t bits) {
  const int E = (int)(bits >> 23) & 0xFF;
  if (E == 0) return -127;
  const int e = (E - 127) - 8 + (((bits & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

MPM_DEV float pow2_neg(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// max of two pairs of bf16 magnitudes, half by half; of a number and a NaN the
// number
MPM_DEV uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
// max |x| of the low and of the high halves of bf16 pairs, with packed bf16 abs / max
template <int N>
MPM_DEV uint32_t absmax_bf16x2_halves(const uint32_t (&w)[N]) {
  __nv_bfloat162 acc = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
  for (int j = 1; j < N; ++j) acc = __hmax2(acc, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));
  return *reinterpret_cast<uint32_t*>(&acc);
}
// the larger half, by its bits: of a number and a NaN (a half that held nothing
// else) the NaN
MPM_DEV uint32_t larger_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
// max |x| over bf16 pairs, as the 16-bit pattern of the larger magnitude in the
// low half
template <int N>
MPM_DEV uint32_t absmax_bf16x2_packed(const uint32_t (&w)[N]) { return larger_half(absmax_bf16x2_halves(w)); }

}  // namespace mpm
