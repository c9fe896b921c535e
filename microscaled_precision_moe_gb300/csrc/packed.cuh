// Two fp32 operations in one instruction, each half the IEEE result of the
// scalar one (the products are mul_f32x2 in common.cuh).
#pragma once
#include "common.cuh"

namespace mpm {

MPM_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MPM_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// a pair of bf16 as two fp32
MPM_DEV uint64_t widen2(uint32_t w) { return f32x2(bf16lo(w), bf16hi(w)); }

}  // namespace mpm
