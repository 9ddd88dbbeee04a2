// kvq.hip -- writing rows of keys and values into the coded cache and reading them
// back.  A row (the head_dim values of one token and one cache head) becomes signed
// levels of its own largest magnitude, to nearest:
//   scale = amax / L,  code = z + rint(x * L / amax),  L = 2^(bits-1) - 1, z = 2^(bits-1).
// Both are bound by HBM: a row is read once and written once.  Measured with nothing in
// the caches, launch included (about 5 us): 16384 tokens of 8 heads of 128 from bf16 to
// 4 bits 21.9 us (85 MB), back 20.1 us; 32768 tokens read back from 8 bits 39.1 us (204
// MB).  A large copy runs at 4.8 TB/s.
//
// A lane holds eight consecutive values, so a row takes head_dim / 8 lanes of a wave
// and its maximum a few lane exchanges.  A workgroup takes consecutive tokens of one
// head: the input rows of a head are far apart anyway (each a whole number of cache
// lines), while the codes and scales of neighbouring tokens are neighbours in a page.
#include "kvq_common.h"

namespace onebit {

constexpr int kKvqBlock = 256;
constexpr int kKvqRows = 4;  // of a thread

// Rows whose largest magnitude is below this are stored as zeros: L / amax stays far
// from overflow, and every scale that is not 0 is a normal number.
constexpr float kKvqTiny = 0x1p-110f;

struct KvqWriteArgs {
    KvqCache c;
    const void *src[2];
    int64_t token_stride[2];
    int64_t head_stride[2];
    const int64_t *slots;
    int64_t tokens;
};

struct KvqReadArgs {
    KvqCache c;
    void *dst[2];
    const int64_t *slots;
    int64_t tokens;
};

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

template <int GT>
__device__ __forceinline__ void load8(const void *p, int64_t i, float (&f)[8]) {
    if (GT == kGradF32) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = s[0], b = s[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        // (whole cache lines, read once: the streaming policy)
        const uint4 h = ld_stream(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
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

// The cache rows of a thread's rows, STEP apart; the head's first for those to be skipped.  All
// slots are asked for at once and without a branch (the last one in place of those
// behind it): the compiler would wait for each where the ways join.
template <int STEP>
__device__ __forceinline__ void cache_rows(const KvqCache &c, const int64_t *slots, int64_t first, int64_t tokens, int h,
                                           int64_t (&row)[kKvqRows], bool (&ok)[kKvqRows]) {
    int64_t slot[kKvqRows];
#pragma unroll
    for (int r = 0; r < kKvqRows; ++r) slot[r] = slots[min(first + r * STEP, tokens - 1)];
#pragma unroll
    for (int r = 0; r < kKvqRows; ++r) {
        ok[r] = (first + r * STEP < tokens) & (slot[r] >= 0) & (slot[r] < c.n_slots);
        const int64_t at = ok[r] ? slot[r] : 0;
        row[r] = ((at >> c.shift) * c.heads + h) * c.page + (int32_t)(at & (c.page - 1));
    }
}

template <int GT, int D, int BITS>
__global__ __launch_bounds__(kKvqBlock) void k_kvq_quantize(KvqWriteArgs a) {
    constexpr int kLanes = D / 8, kRows = kKvqBlock / kLanes;
    const int sub = threadIdx.x % kLanes;
    const int h = blockIdx.y >> 1, kv = blockIdx.y & 1;
    const int64_t first = (int64_t)blockIdx.x * (kKvqRows * kRows) + threadIdx.x / kLanes;
    int64_t row[kKvqRows];
    bool ok[kKvqRows];
    float f[kKvqRows][8];
    cache_rows<kRows>(a.c, a.slots, first, a.tokens, h, row, ok);
#pragma unroll
    for (int r = 0; r < kKvqRows; ++r) {
        // (a row that is skipped reads the call's first one)
        const int64_t i = ok[r] ? first + r * kRows : 0;
        load8<GT>(a.src[kv], i * a.token_stride[kv] + h * a.head_stride[kv] + 8 * sub, f[r]);
    }
#pragma unroll
    for (int r = 0; r < kKvqRows; ++r) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(f[r][k]) & 0x7fffffffu);
        top = max_over_lanes<kLanes>(top);  // the order of magnitudes, infinity and NaN above all others
        if (!ok[r]) continue;
        const float amax = __uint_as_float(top);
        const bool finite = top < 0x7f800000u, live = finite && amax >= kKvqTiny;
        const float L = (float)KvqLevels<BITS>::kTop;
        const float inv = __fdiv_rn(L, live ? amax : L);
        const float scale = live ? fminf(__fdiv_rn(amax, L), KvqLevels<BITS>::kMaxScale)
                                 : finite ? 0.0f : __uint_as_float(0x7fc00000u);
        uint32_t c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) c[k] = code_bits<BITS>(f[r][k], inv);
        if (BITS == 8) {
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t lo = __builtin_amdgcn_perm(c[4 * k + 1], c[4 * k], 0x0c0c0400u);
                const uint32_t hi = __builtin_amdgcn_perm(c[4 * k + 3], c[4 * k + 2], 0x0c0c0400u);
                w[k] = live ? lo | (hi << 16) : 0x80808080u;
            }
            *reinterpret_cast<uint2 *>(a.c.codes[kv] + row[r] * D + 8 * sub) = make_uint2(w[0], w[1]);
        } else {
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) w |= (c[k] & 15u) << (4 * k);
            *reinterpret_cast<uint32_t *>(a.c.codes[kv] + row[r] * (D / 2) + 4 * sub) = live ? w : 0x88888888u;
        }
        if (sub == 0) a.c.scales[kv][row[r]] = scale;
    }
}

template <int GT, int D, int BITS>
__global__ __launch_bounds__(kKvqBlock) void k_kvq_dequantize(KvqReadArgs a) {
    constexpr int kLanes = D / 8, kRows = kKvqBlock / kLanes;
    const int sub = threadIdx.x % kLanes;
    const int h = blockIdx.y >> 1, kv = blockIdx.y & 1;
    const int64_t first = (int64_t)blockIdx.x * (kKvqRows * kRows) + threadIdx.x / kLanes;
    int64_t row[kKvqRows];
    bool ok[kKvqRows];
    uint32_t w[kKvqRows][2];
    float scale[kKvqRows];
    cache_rows<kRows>(a.c, a.slots, first, a.tokens, h, row, ok);
#pragma unroll
    for (int r = 0; r < kKvqRows; ++r) {
        scale[r] = a.c.scales[kv][row[r]];
        if (BITS == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(a.c.codes[kv] + row[r] * D + 8 * sub);
            w[r][0] = v.x;
            w[r][1] = v.y;
        } else {
            w[r][0] = *reinterpret_cast<const uint32_t *>(a.c.codes[kv] + row[r] * (D / 2) + 4 * sub);
        }
    }
#pragma unroll
    for (int r = 0; r < kKvqRows; ++r) {
        if (!ok[r]) continue;
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t c = BITS == 8 ? (w[r][k >> 2] >> (8 * (k & 3))) & 255u : (w[r][0] >> (4 * k)) & 15u;
            y[k] = mul_rn(sub_rn((float)(int)c, (float)KvqLevels<BITS>::kZero), scale[r]);
        }
        const int64_t o = ((first + r * kRows) * a.c.heads + h) * D + 8 * sub;
        if (GT == kGradF32) {
            float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.dst[kv]) + o);
            d[0] = make_float4(y[0], y[1], y[2], y[3]);
            d[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dst[kv]) + o) =
                make_uint4(round_pair<GT>(y[0], y[1]), round_pair<GT>(y[2], y[3]), round_pair<GT>(y[4], y[5]),
                           round_pair<GT>(y[6], y[7]));
        }
    }
}

template <int D>
static dim3 kvq_grid(int64_t tokens, int heads) {
    constexpr int64_t each = (int64_t)kKvqRows * (kKvqBlock / (D / 8));
    return dim3((unsigned)((tokens + each - 1) / each), 2 * heads);
}
template <int GT, int D, int BITS>
static void launch_write(const KvqWriteArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((k_kvq_quantize<GT, D, BITS>), kvq_grid<D>(a.tokens, a.c.heads), dim3(kKvqBlock), 0, s, a);
}
template <int GT, int D, int BITS>
static void launch_read(const KvqReadArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((k_kvq_dequantize<GT, D, BITS>), kvq_grid<D>(a.tokens, a.c.heads), dim3(kKvqBlock), 0, s, a);
}

// f.run<type, head_dim, bits>() for the runtime values
template <int GT, int D, typename F>
static void kvq_dispatch_bits(int bits, F f) {
    if (bits == 4)
        f.template run<GT, D, 4>();
    else
        f.template run<GT, D, 8>();
}
template <int GT, typename F>
static void kvq_dispatch_dim(int dim, int bits, F f) {
    if (dim == 64)
        kvq_dispatch_bits<GT, 64>(bits, f);
    else if (dim == 128)
        kvq_dispatch_bits<GT, 128>(bits, f);
    else
        kvq_dispatch_bits<GT, 256>(bits, f);
}
template <typename F>
static void kvq_dispatch(onebit_dtype_t dtype, int dim, int bits, F f) {
    if (dtype == ONEBIT_F32)
        kvq_dispatch_dim<kGradF32>(dim, bits, f);
    else if (dtype == ONEBIT_BF16)
        kvq_dispatch_dim<kGradBF16>(dim, bits, f);
    else
        kvq_dispatch_dim<kGradF16>(dim, bits, f);
}
struct WriteLaunch {
    const KvqWriteArgs &a;
    hipStream_t s;
    template <int GT, int D, int BITS>
    void run() const { launch_write<GT, D, BITS>(a, s); }
};
struct ReadLaunch {
    const KvqReadArgs &a;
    hipStream_t s;
    template <int GT, int D, int BITS>
    void run() const { launch_read<GT, D, BITS>(a, s); }
};

// Checks shared by both calls.  The grid has ceil(tokens / rows) x 2 heads workgroups
// of at least 32 rows: fewer than 2^32 threads along x, at most 65535 workgroups along y.
static onebit_status_t kvq_check_rows(const kvq_cache_t *cache, onebit_dtype_t dtype, int64_t tokens, KvqCache *out) {
    if (dtype != ONEBIT_F32 && dtype != ONEBIT_BF16 && dtype != ONEBIT_F16) return ONEBIT_ERR_INVALID;
    if (tokens < 0 || tokens >= (1 << 26)) return ONEBIT_ERR_INVALID;
    return kvq_check_cache(cache, out);
}

}  // namespace onebit

using namespace onebit;

extern "C" onebit_status_t kvq_quantize(const void *k, const void *v, onebit_dtype_t dtype, int64_t tokens,
                                        int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                        int64_t v_head_stride, const int64_t *slots, const kvq_cache_t *cache,
                                        void *stream) {
    KvqWriteArgs a{};
    const onebit_status_t st = kvq_check_rows(cache, dtype, tokens, &a.c);
    if (st != ONEBIT_OK) return st;
    if (tokens == 0) return ONEBIT_OK;
    if (!k || !v || !slots) return ONEBIT_ERR_INVALID;
    const int64_t unit = dtype == ONEBIT_F32 ? 4 : 8;  // elements in 16 bytes
    if (!aligned16(k) || !aligned16(v) || !aligned_to(slots, 8) || k_token_stride % unit || k_head_stride % unit ||
        v_token_stride % unit || v_head_stride % unit)
        return ONEBIT_ERR_ALIGN;
    a.src[0] = k;
    a.src[1] = v;
    a.token_stride[0] = k_token_stride;
    a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride;
    a.head_stride[1] = v_head_stride;
    a.slots = slots;
    a.tokens = tokens;
    if (a.c.n_slots == 0) return ONEBIT_OK;  // every slot is outside the cache
    kvq_dispatch(dtype, cache->head_dim, cache->bits, WriteLaunch{a, static_cast<hipStream_t>(stream)});
    return hip_status(hipGetLastError());
}

extern "C" onebit_status_t kvq_dequantize(const kvq_cache_t *cache, const int64_t *slots, int64_t tokens, void *k_out,
                                          void *v_out, onebit_dtype_t out_dtype, void *stream) {
    KvqReadArgs a{};
    const onebit_status_t st = kvq_check_rows(cache, out_dtype, tokens, &a.c);
    if (st != ONEBIT_OK) return st;
    if (tokens == 0) return ONEBIT_OK;
    if (!k_out || !v_out || !slots) return ONEBIT_ERR_INVALID;
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned_to(slots, 8)) return ONEBIT_ERR_ALIGN;
    a.dst[0] = k_out;
    a.dst[1] = v_out;
    a.slots = slots;
    a.tokens = tokens;
    if (a.c.n_slots == 0) return ONEBIT_OK;  // every slot is outside the cache
    kvq_dispatch(out_dtype, cache->head_dim, cache->bits, ReadLaunch{a, static_cast<hipStream_t>(stream)});
    return hip_status(hipGetLastError());
}
