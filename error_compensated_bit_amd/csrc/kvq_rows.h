// kvq_rows.h -- rows of keys and values on their way into the coded cache: loads,
// the code of a row, and the choice of an instantiation, shared by the calls that write
// them (kvq.hip, kvq_append.hip).
#pragma once

#include "kvq_common.h"

namespace onebit {

// Rows whose largest magnitude is below this are stored as zeros: L / amax stays far
// from overflow, and every scale that is not 0 is a normal number.
constexpr float kKvqTiny = 0x1p-110f;

// maximum over each aligned group of LANES lanes (8, 16 or 32)
template <int LANES>
__device__ __forceinline__ uint32_t max_over_lanes(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
    if (LANES >= 16) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // row_mirror
    if (LANES >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    return v;
}

// values i .. i + 7; STREAM: 16-bit ones are read once, as whole cache lines
template <int GT, bool STREAM = true>
__device__ __forceinline__ void load8(const void *p, int64_t i, float (&f)[8]) {
    if (GT == kGradF32) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = s[0], b = s[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        const uint4 h = STREAM ? ld_stream(s) : *s;
        const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = half_bits_to_float<GT>(w[k] & 0xffffu);
            f[2 * k + 1] = half_bits_to_float<GT>(w[k] >> 16);
        }
    }
}

// x * inv + (1.5 * 2^23 + z): the sum's last bit has weight 1, so the one rounding of
// the fused operation rounds the exact product to an integer, ties to even (1.5 * 2^23
// and z are even), and the low byte of the result is the code.
template <int BITS>
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
    return __float_as_uint(__fmaf_rn(x, inv, 12582912.0f + (float)KvqLevels<BITS>::kZero));
}

// One row's codes and scale, written to cache row `row` (ok: else nothing is written): f holds
// values 8 sub .. 8 sub + 7 of the row, D / 8 lanes hold the row, and all of them call.
template <int D, int BITS>
__device__ __forceinline__ void code_row(const KvqCache &c, int kv, const float (&f)[8], int64_t row, int sub, bool ok) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(f[k]) & 0x7fffffffu);
    top = max_over_lanes<D / 8>(top);  // the order of magnitudes, infinity and NaN above all others
    if (!ok) return;
    const float amax = __uint_as_float(top);
    const bool finite = top < 0x7f800000u, live = finite && amax >= kKvqTiny;
    const float L = (float)KvqLevels<BITS>::kTop;
    const float inv = __fdiv_rn(L, live ? amax : L);
    const float scale = live ? fminf(__fdiv_rn(amax, L), KvqLevels<BITS>::kMaxScale)
                             : finite ? 0.0f : __uint_as_float(0x7fc00000u);
    uint32_t code[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) code[k] = code_bits<BITS>(f[k], inv);
    if (BITS == 8) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t lo = __builtin_amdgcn_perm(code[4 * k + 1], code[4 * k], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(code[4 * k + 3], code[4 * k + 2], 0x0c0c0400u);
            w[k] = live ? lo | (hi << 16) : 0x80808080u;
        }
        *reinterpret_cast<uint2 *>(c.codes[kv] + row * D + 8 * sub) = make_uint2(w[0], w[1]);
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) w |= (code[k] & 15u) << (4 * k);
        *reinterpret_cast<uint32_t *>(c.codes[kv] + row * (D / 2) + 4 * sub) = live ? w : 0x88888888u;
    }
    if (sub == 0) c.scales[kv][row] = scale;
}

// f.run<type, head_dim, bits>() for the runtime values
template <int GT, int D, typename F>
inline void kvq_dispatch_bits(int bits, F f) {
    if (bits == 4)
        f.template run<GT, D, 4>();
    else
        f.template run<GT, D, 8>();
}
template <int GT, typename F>
inline void kvq_dispatch_dim(int dim, int bits, F f) {
    if (dim == 64)
        kvq_dispatch_bits<GT, 64>(bits, f);
    else if (dim == 128)
        kvq_dispatch_bits<GT, 128>(bits, f);
    else
        kvq_dispatch_bits<GT, 256>(bits, f);
}
template <typename F>
inline void kvq_dispatch(onebit_dtype_t dtype, int dim, int bits, F f) {
    if (dtype == ONEBIT_F32)
        kvq_dispatch_dim<kGradF32>(dim, bits, f);
    else if (dtype == ONEBIT_BF16)
        kvq_dispatch_dim<kGradBF16>(dim, bits, f);
    else
        kvq_dispatch_dim<kGradF16>(dim, bits, f);
}

// Checks shared by the calls over rows.  They bound the grids: kvq_quantize and kvq_dequantize have
// ceil(tokens / rows) x 2 heads workgroups of at least 32 rows, kvq_append is bounded at its own launch.
inline onebit_status_t kvq_check_rows(const kvq_cache_t *cache, onebit_dtype_t dtype, int64_t tokens, KvqCache *out) {
    if (dtype != ONEBIT_F32 && dtype != ONEBIT_BF16 && dtype != ONEBIT_F16) return ONEBIT_ERR_INVALID;
    if (tokens < 0 || tokens >= (1 << 26)) return ONEBIT_ERR_INVALID;
    return kvq_check_cache(cache, out);
}

}  // namespace onebit
