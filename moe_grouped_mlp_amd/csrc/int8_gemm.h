#pragma once

// What the two kernels of the 8-bit integer product share.  Tiles, their order
// and the operands' way into LDS are those of the FP8 product.
#include "fp8_gemm_kernel.h"

namespace moe {
namespace {

constexpr int kInt8Blk = kFp8Blk;   // K bytes of a stage

// D = A . B + C over 64 values of K: a lane's 16 codes are those of row
// (lane % 16) of either operand, at 16 (lane / 16).
MOE_DEV i32x4 int8_mfma(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// A sum rounded to fp32 once and scaled there.
MOE_DEV float int8_scaled(int sum, float a, float b) { return static_cast<float>(sum) * a * b; }

}  // namespace
}  // namespace moe
