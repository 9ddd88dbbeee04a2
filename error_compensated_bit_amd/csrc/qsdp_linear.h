// qsdp_linear.h -- what the kernels of the products with coded weights share.
#pragma once

#include <hip/hip_runtime.h>

#include "kvq_attention.h"

namespace onebit {

struct LinearArgs {
    const uint8_t *codes;
    const float *lo, *hi;
    int64_t rows, cols;  // of the matrix
    int32_t bucket;
    // ceil(2^32 / (bucket / 32)): i / (bucket / 32) is the upper half of i times it for i < 2^21 (it is off by
    // less than 2^11 / 2^32 of i), if the bucket has more than 32 values
    uint32_t bucket_magic;
    const uint16_t *x;  // [tokens][depth]
    int64_t x_stride;
    uint16_t *out;  // [tokens][width]
    int64_t out_stride;
    int64_t tokens;
    void *workspace;
};

typedef __bf16 bf16x8_v __attribute__((ext_vector_type(8)));

template <int GT>
__device__ __forceinline__ f32x4_v product16(const u32x4_v a, const u32x4_v b, f32x4_v c) {
    if (GT == kGradBF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_v, a), __builtin_bit_cast(bf16x8_v, b), c,
                                                       0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_v, a), __builtin_bit_cast(f16x8_v, b), c, 0, 0, 0);
}

// The bucket of the flat vector's 32-value part p (p < 2^43), and the part's place in it.
struct Bucket {
    int64_t index;
    uint32_t part;
};
__device__ __forceinline__ Bucket bucket_of(int64_t p, uint32_t bucket_parts) {
    // the quotient in binary64 is off by one at most
    int64_t q = (int64_t)((double)p * (1.0 / (double)bucket_parts));
    int64_t r = p - q * bucket_parts;
    if (r < 0) {
        --q;
        r += bucket_parts;
    } else if (r >= bucket_parts) {
        ++q;
        r -= bucket_parts;
    }
    return {q, (uint32_t)r};
}

// fl32(fl32(hi - lo) / (2^BITS - 1)): the product with the rounded reciprocal, corrected once by its
// exact remainder, is the correctly rounded quotient (Markstein).  A range that is not finite
// gives NaN.
template <int BITS>
__device__ __forceinline__ float bucket_delta(float lo, float hi) {
    constexpr float kLevels = (float)((1 << BITS) - 1), kInv = 1.0f / kLevels;
    const float range = sub_rn(hi, lo), q = mul_rn(range, kInv);
    return __fmaf_rn(__fmaf_rn(-q, kLevels, range), kInv, q);
}

}  // namespace onebit
