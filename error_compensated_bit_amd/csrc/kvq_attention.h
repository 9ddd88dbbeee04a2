// kvq_attention.h -- what the attention kernels over the coded cache share: their
// arguments, the sequences' bounds, the expansion of codes into matrix operands, the
// queries' operand and the softmax's scores.
//
// Codes enter the matrix cores as they are.  A byte c in the low half of a 16-bit
// word is, read as fp16, the subnormal number c * 2^-24: exact, and one byte
// permutation makes two of them.  Scores are sums over codes; what the definition
// subtracts and scales stays outside of the sum:
//   <q, k_j> = ks_j (<q, c_j> - z sum_d q_d).
// (The matrix cores align the products by the operands' exponent fields, where all
// subnormal numbers count as 2^-14: a product is summed as exactly as if its code were
// 1024, eight times the largest magnitude.  A 4-bit code is put into the byte's high
// nibble; in the low one it would lose four bits more.)  Values, whose sum is over
// thousands of tokens and may come out far smaller than the codes' offset z, enter as
// (c - z) 2^-9, exact too, one fused operation more for two of them.
#pragma once

#include "kvq_common.h"

namespace onebit {

typedef _Float16 f16x8_v __attribute__((ext_vector_type(8)));
typedef float f32x4_v __attribute__((ext_vector_type(4)));
typedef float f32x16_v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_v __attribute__((ext_vector_type(4)));

// the value of code 1 as an operand is 2^-kCodeShift
template <int BITS>
constexpr int kCodeShift = BITS == 8 ? 24 : 20;

constexpr float kNone = -3.40282347e+38f;  // running maximum before the first key

struct KvqAttnArgs {
    KvqCache c;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t q_token_stride, q_head_stride;
    const int32_t *q_offsets;  // of the first sequence of this launch; null: q_uniform rows each
    const int32_t *kv_lens;
    const int32_t *table;
    int64_t table_stride;
    int32_t batch, total_q, q_heads, group;
    int32_t q_first;     // first row of this launch's first sequence where q_offsets is null
    int32_t q_uniform;
    int32_t max_tokens;  // max_pages * page
    int32_t max_rows;    // most rows (tokens x group) of a sequence that the step kernel takes
    int32_t window;
    float scale2;        // |sm_scale| * log2(e)
    uint32_t q_sign;     // sign bit to flip in q where sm_scale is negative
    float cap2;          // softcap * log2(e); 0: none
    float cap_scale;     // 2 / softcap: tanh(s / cap) from exp2(cap_scale * s * log2(e))
    void *workspace;
};

// Rows and cached tokens of sequence b; out-of-range numbers are clamped.
struct KvqSeq {
    int32_t q0, len, kv;
};
__device__ __forceinline__ KvqSeq kvq_seq(const KvqAttnArgs &a, int b) {
    KvqSeq s;
    if (a.q_offsets) {
        s.q0 = min(max(a.q_offsets[b], 0), a.total_q);
        s.len = max(min(a.q_offsets[b + 1], a.total_q) - s.q0, 0);
    } else {
        s.q0 = a.q_first + b * a.q_uniform;
        s.len = a.q_uniform;
    }
    s.kv = min(max(a.kv_lens[b], 0), a.max_tokens);
    return s;
}

// Positions [lo, hi) that query t of the sequence attends to (hi <= lo: none).
__host__ __device__ __forceinline__ int kvq_hi(const KvqSeq &s, int t) { return max(s.kv - s.len + t + 1, 0); }
__host__ __device__ __forceinline__ int kvq_lo(const KvqAttnArgs &a, const KvqSeq &s, int t) {
    const int p = s.kv - s.len + t;
    return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

// Four consecutive outputs, rounded to their type.
template <int GT>
__device__ __forceinline__ void store_out4(uint16_t *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(round_pair<GT>(v[0], v[1]), round_pair<GT>(v[2], v[3]));
}

// Eight codes of consecutive dimensions as an operand of a product over dimensions.
// 8 bits: from two words; the operand's elements are in order.  4 bits: from one word;
// elements 0 4, 1 5, 2 6, 3 7 of the eight.
template <int BITS>
__device__ __forceinline__ f16x8_v codes_over_dims(uint32_t w0, uint32_t w1) {
    u32x4_v r;
    if (BITS == 8) {
        r.x = __builtin_amdgcn_perm(0u, w0, 0x0c010c00u);
        r.y = __builtin_amdgcn_perm(0u, w0, 0x0c030c02u);
        r.z = __builtin_amdgcn_perm(0u, w1, 0x0c010c00u);
        r.w = __builtin_amdgcn_perm(0u, w1, 0x0c030c02u);
    } else {
        r.x = (w0 << 4) & 0x00f000f0u;
        r.y = w0 & 0x00f000f0u;
        r.z = (w0 >> 4) & 0x00f000f0u;
        r.w = (w0 >> 8) & 0x00f000f0u;
    }
    return __builtin_bit_cast(f16x8_v, r);
}

// The matching operand of eight consecutive query values, scaled by `up`, a power of two.
template <int BITS>
__device__ __forceinline__ f16x8_v query_operand(const float (&q)[8], float up) {
    u32x4_v r;
    if (BITS == 8) {
        r.x = round_pair<kGradF16>(q[0] * up, q[1] * up);
        r.y = round_pair<kGradF16>(q[2] * up, q[3] * up);
        r.z = round_pair<kGradF16>(q[4] * up, q[5] * up);
        r.w = round_pair<kGradF16>(q[6] * up, q[7] * up);
    } else {
        r.x = round_pair<kGradF16>(q[0] * up, q[4] * up);
        r.y = round_pair<kGradF16>(q[1] * up, q[5] * up);
        r.z = round_pair<kGradF16>(q[2] * up, q[6] * up);
        r.w = round_pair<kGradF16>(q[3] * up, q[7] * up);
    }
    return __builtin_bit_cast(f16x8_v, r);
}

// Codes of one dimension (number u of the lane's consecutive ones) of two tokens whose
// words are wa and wb.
template <int BITS>
__device__ __forceinline__ uint32_t code_pair(uint32_t wa, uint32_t wb, int u) {
    if (BITS == 8) {
        const uint32_t byte = u & 3;
        return __builtin_amdgcn_perm(wb, wa, 0x0c040c00u + byte * 0x00010001u);
    }
    const uint32_t byte = (u >> 1) & 3;
    const uint32_t x = __builtin_amdgcn_perm(wb, wa, 0x0c040c00u + byte * 0x00010001u);
    return ((u & 1) ? x : x << 4) & 0x00f000f0u;
}

// Weights are rounded to fp16 (11 bits) for the matrix cores.  For bf16 outputs that is
// an eighth of the output's own rounding; an fp16 output would come out 1.6 times as
// far off (measured), so there what the rounding drops goes through the matrix cores
// as a second fp16 operand.
template <int GT>
constexpr bool kTwoPart = GT == kGradF16;

__device__ __forceinline__ uint32_t rest_pair(float a, float b, uint32_t pair) {
    const f16x2_v h = __builtin_bit_cast(f16x2_v, pair);
    // both differences are exact (the compiler makes a conversion and a subtraction of each)
    return round_pair<kGradF16>(fmaf((float)h[0], -1.0f, a), fmaf((float)h[1], -1.0f, b));
}

__device__ __forceinline__ f16x2_v splat16(float v) {
    const _Float16 h = (_Float16)v;
    return (f16x2_v){h, h};
}
__device__ __forceinline__ uint32_t fma16(uint32_t codes, f16x2_v scale, f16x2_v offset) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2_v, codes), scale, offset));
}

// A code operand times kUnitScale, less kUnitOffset: (c - z) 2^-kUnitShift, exactly, in one
// fused operation for two.
template <int BITS>
constexpr float kUnitScale = BITS == 8 ? 0x1p15f : 0x1p11f;
// z as an operand is 2^-17 at either width
template <int BITS>
constexpr float kUnitOffset = kUnitScale<BITS> * 0x1p-17f;
constexpr int kUnitShift = 9;

// Exponent k that brings a row of queries whose largest magnitude is amax to
// [2^14, 2^15) as fp16: exact for bf16 and fp16 values down to 2^-29 of the largest,
// and smaller ones are off by less than 2^-39 of it.
__device__ __forceinline__ int query_exponent(float amax) {
    const int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127;  // zero and subnormal: -127
    return min(14 - e, 120);
}

// a / b for a >= 0, b > 0: the 64-bit division only where it is needed
__device__ __forceinline__ int64_t udiv(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// the value every lane of the wave holds, as a scalar
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(127 + k) << 23); }  // -126 <= k <= 127

// softcap * tanh(s / softcap) in units of log2(e), from y = 2 log2(e) s / softcap.  The
// difference is off by 2^-21 of the cap, whatever the score: caps above 64 (kWideCap2 in
// these units) take scores below an eighth of the cap from tanh's series, whose first
// term left out is 2^-29 of the score.
constexpr float kWideCap2 = 92.4f;
__device__ __forceinline__ float capped(float y, float cap2) {
    return fmaf(-2.0f * cap2, __builtin_amdgcn_rcpf(exp2_fast(y) + 1.0f), cap2);
}
__device__ __forceinline__ float capped_wide(float y, float cap2) {
    const float z = y * 0.346573590f, zz = z * z;
    const float series = fmaf(zz, fmaf(zz, fmaf(zz, -17.0f / 315, 2.0f / 15), -1.0f / 3), 1.0f);
    return fabsf(z) < 0.125f ? cap2 * (z * series) : capped(y, cap2);
}

// Largest power of two k with |s| 2^k < 2^7 for every value scale up to `top`.
__device__ __forceinline__ int value_exponent(float top) {
    const int e = (int)((__float_as_uint(top) >> 23) & 255u) - 126;  // top < 2^e
    return min(max(7 - e, -126), 126);
}

}  // namespace onebit
