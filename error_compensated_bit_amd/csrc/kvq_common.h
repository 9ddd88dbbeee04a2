// kvq_common.h -- the coded key/value cache: its layout on the device and the checks
// shared by the calls that write it, read it back and attend to it (kvq.hip,
// kvq_attention.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "internal.h"
#include "onebit.h"

namespace onebit {

// One pair of pools (codes, scales).  Row r = (page number * heads + head) * page +
// offset has its codes at r * row_bytes and its scale at r.
struct KvqCache {
    uint8_t *codes[2];  // 0 keys, 1 values
    float *scales[2];
    int64_t n_pages;
    int64_t n_slots;  // n_pages * page
    int32_t heads;
    int32_t page;
    int32_t shift;  // log2(page)
};

template <int BITS>
struct KvqLevels {
    static constexpr int kTop = (1 << (BITS - 1)) - 1;  // L
    static constexpr int kZero = 1 << (BITS - 1);       // z
    // the largest fp32 number with L times it finite: amax / L rounded up can pass it
    static constexpr float kMaxScale = BITS == 8 ? 0x1.020406p+121f : 0x1.249248p+125f;
};

typedef float f32x2_v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_v __attribute__((ext_vector_type(2)));

// two fp32 values rounded to nearest even, first in the low half
template <int GT>
__device__ __forceinline__ uint32_t round_pair(float a, float b) {
    const f32x2_v v = {a, b};
    if (GT == kGradBF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_v));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_v));
}

// Checks of a caller's cache; fills *out.  Pointers are needed only where there are pages.
inline onebit_status_t kvq_check_cache(const kvq_cache_t *c, KvqCache *out) {
    if (!c) return ONEBIT_ERR_INVALID;
    if (c->bits != 4 && c->bits != 8) return ONEBIT_ERR_INVALID;
    if (c->kv_heads < 1 || c->kv_heads > 32767 || c->n_pages < 0 || c->page < 16 || c->page > 1024 || (c->page & (c->page - 1)))
        return ONEBIT_ERR_INVALID;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return ONEBIT_ERR_UNSUPPORTED;
    if (c->n_pages >= (int64_t{1} << 47) / c->page) return ONEBIT_ERR_INVALID;
    if (c->n_pages > 0) {
        if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return ONEBIT_ERR_INVALID;
        if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
            return ONEBIT_ERR_ALIGN;
    }
    out->codes[0] = c->k_codes;
    out->codes[1] = c->v_codes;
    out->scales[0] = c->k_scales;
    out->scales[1] = c->v_scales;
    out->n_pages = c->n_pages;
    out->n_slots = c->n_pages * c->page;
    out->heads = c->kv_heads;
    out->page = c->page;
    out->shift = __builtin_ctz((unsigned)c->page);
    return ONEBIT_OK;
}

}  // namespace onebit
