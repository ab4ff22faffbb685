// Shared by the FP8 block-128 kernels: the block size and bf16 pair rounding.
#pragma once

#include "common.h"

namespace nvfp4moe {

constexpr int kFp8Block = FP8_BLOCK;   // elements that share one scale, along K (and along N for weights)

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// two floats -> two bf16 in one word (a in the low half), nearest even, NaN kept
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}

}  // namespace nvfp4moe
