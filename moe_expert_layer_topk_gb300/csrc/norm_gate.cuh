// What the norm after a block and its backward share: the gate and argument checks.
#pragma once

#include "norm.cuh"

namespace moe {

// sigmoid(x) and its derivative, from e^-|x|: neither loses digits at either end.
struct Gate {
  float g, d;
};
// e^-|x| = 2^(-|x| log2 e) by the approximate instructions: each is off by 2^-22 or so, what is
// below 2^-126 is 0, and the rounding of the exponent adds |x| 2^-24 (1e-6 at a logit of -20;
// at +20 it is lost beside 1).
__device__ __forceinline__ Gate sigmoid(float x) {
  float e, t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(x) * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(1.0f + e));
  return {x >= 0.f ? t : e * t, e * t * t};
}

inline int check_post(const char* fn, int T, int H, int fp32, int norm, int gate_kind) {
  if (int rc = check_norm(fn, T, H, fp32)) return rc;
  if ((norm != 0 && norm != 1) || gate_kind < 0 || gate_kind > 2)
    return fail(MOE_ERR_INVALID_ARG, "%s: need norm 0 or 1, gate_kind 0, 1 or 2", fn);
  return MOE_OK;
}

inline bool gate_aligned(int kind, const void* gate) {
  return kind == 2 ? aligned16(gate) : (reinterpret_cast<uintptr_t>(gate) & 3u) == 0;
}

}  // namespace moe
