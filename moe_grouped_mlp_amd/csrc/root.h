#pragma once

namespace moe {

// The root of v in [2^-96, 2^128) from y, the hardware's reciprocal root, which is
// off by an ulp at most: one Newton step, with the residual in a fused multiply-add.
// Correctly rounded: all significands of either parity were tried with every y
// within an ulp, and one of them is rounded wrongly by one y, 0x406e9372 (3.727...)
// by the one above the true value by 0.85 ulp.  The hardware gives the other there,
// whatever the exponent.  (A Newton step for both before this one would serve every y:
// 705 M elements with 8-bit states 1242 us, with this 1228.)
__host__ __device__ inline float root_from(float v, float y) {
  const float s = v * y;
  return __builtin_fmaf(__builtin_fmaf(-s, s, v), 0.5f * y, s);
}

}  // namespace moe
