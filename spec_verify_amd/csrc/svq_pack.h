// Roundings of pairs, shared by the operators of a tree of drafts.
#pragma once

#include "svq_device.h"

namespace svq {

// Two values as a bf16 pair (nearest even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

}  // namespace svq
