// kvq_append.hip -- new tokens on their way from a projection into attention: queries and
// keys turned by their positions, queries written out, keys and values coded into the cache.
//   a' = a cos - b sin,  b' = b cos + a sin     for each pair (a, b) of a head's first values.
// The products of two binary32 numbers are exact in binary64 and their sum is rounded
// there once, then to binary32: the turned values, and with them the codes, do not
// depend on the order or fusing of the operations.
//
// Bound by HBM: a token's queries, keys and values are read once, its queries and codes
// written once.  A lane holds eight consecutive values of a head, as in kvq_quantize; it takes
// the same place of kAppendHeads heads, so that the cosines and sines, four times a row's
// bytes, are read once for them.
//
// Measured: 16384 tokens of 32 + 2 x 8 heads of 128, bf16, 4 bits, 83 to 90 us for 362 MB (4.0 to 4.4 TB/s;
// a copy moves 4.8), fp32 164 us for 698 MB; 5003 of 16 + 2 x 16 heads of 64, fp16, 8 bits, 13.6 us; 64 tokens 5.3
// us (fp32 4.8, in a graph).
#include "kvq_rows.h"

namespace onebit {

constexpr int kAppendBlock = 256;
constexpr int kAppendHeads = 4;  // of a thread

struct KvqAppendArgs {
    KvqCache c;
    const void *src[3];  // queries, keys, values
    int64_t token_stride[3];
    int64_t head_stride[3];
    void *out;  // turned queries
    int64_t out_token_stride;
    int64_t out_head_stride;
    const int64_t *positions;
    const int64_t *slots;
    const float *rotary;
    int64_t max_position;
    int64_t tokens;
    int32_t q_heads;
    int32_t rot;
    int32_t interleaved;
};

template <int GT, int D, int BITS>
__global__ __launch_bounds__(kAppendBlock) void k_kvq_append(KvqAppendArgs a) {
    constexpr int kLanes = D / 8, kRows = kAppendBlock / kLanes;
    const int sub = threadIdx.x % kLanes, e = 8 * sub;
    const int64_t mine = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;
    const bool live = mine < a.tokens;
    const int64_t i = live ? mine : a.tokens - 1;
    const int heads = a.q_heads + 2 * a.c.heads, first = blockIdx.y * kAppendHeads;
    const int half = a.rot >> 1;
    const bool turned = e < a.rot, low = e < half;
    const int other = a.interleaved || !turned ? e : low ? e + half : e - half;  // where the pairs' other values begin

    const int64_t position = a.positions[i], slot = a.slots[i];
    float f[kAppendHeads][8], g[kAppendHeads][8];
#pragma unroll
    for (int r = 0; r < kAppendHeads; ++r) {
        // (behind the last head: the last one again, not used)
        const int h = min(first + r, heads - 1);
        const int which = h < a.q_heads ? 0 : h < a.q_heads + a.c.heads ? 1 : 2;
        const int at = which == 0 ? h : which == 1 ? h - a.q_heads : h - a.q_heads - a.c.heads;
        const int64_t row = i * a.token_stride[which] + at * a.head_stride[which];
        load8<GT, false>(a.src[which], row + e, f[r]);
        load8<GT, false>(a.src[which], row + other, g[r]);
    }
    // cosines and signed sines of this lane's values
    double co[8], si[8];
    {
        const bool known = position >= 0 && position < a.max_position;
        const float *t = a.rotary + (known ? position : 0) * a.rot;
        const float nan = __uint_as_float(0x7fc00000u);
        if (a.interleaved) {
            const int j = turned ? e >> 1 : 0;
            const float4 c = *reinterpret_cast<const float4 *>(t + j), s = *reinterpret_cast<const float4 *>(t + half + j);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                co[k] = known ? cc[k >> 1] : nan;
                si[k] = k & 1 ? ss[k >> 1] : -ss[k >> 1];
            }
        } else {
            const int j = !turned ? 0 : low ? e : e - half;
            float cc[8], ss[8];
            load8<kGradF32>(t, j, cc);
            load8<kGradF32>(t, half + j, ss);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                co[k] = known ? cc[k] : nan;
                si[k] = low ? -ss[k] : ss[k];
            }
        }
    }
    // (q_out may be q: rows are read by all of their lanes before one writes)
    __builtin_amdgcn_wave_barrier();
    const bool ok = live && slot >= 0 && slot < a.c.n_slots;
    const int64_t at_page = ok ? slot >> a.c.shift : 0;
    const int32_t in_page = ok ? (int32_t)(slot & (a.c.page - 1)) : 0;
#pragma unroll
    for (int r = 0; r < kAppendHeads; ++r) {
        const int h = first + r;
        if (h >= heads) break;
        if (h < a.q_heads + a.c.heads) {
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float b = a.interleaved ? f[r][k ^ 1] : g[r][k];
                const float v = (float)__fma_rn((double)f[r][k], co[k], __dmul_rn((double)b, si[k]));
                y[k] = turned ? v : f[r][k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) f[r][k] = y[k];
        }
        if (h < a.q_heads) {
            const int64_t o = i * a.out_token_stride + h * a.out_head_stride + e;
            if (!live) {
                // (a row behind the last token)
            } else if (GT == kGradF32) {
                float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o);
                d[0] = make_float4(f[r][0], f[r][1], f[r][2], f[r][3]);
                d[1] = make_float4(f[r][4], f[r][5], f[r][6], f[r][7]);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + o) =
                    make_uint4(round_pair<GT>(f[r][0], f[r][1]), round_pair<GT>(f[r][2], f[r][3]),
                               round_pair<GT>(f[r][4], f[r][5]), round_pair<GT>(f[r][6], f[r][7]));
            }
        } else {
            const int kv = h < a.q_heads + a.c.heads ? 0 : 1;
            const int head = h - a.q_heads - kv * a.c.heads;
            code_row<D, BITS>(a.c, kv, f[r], (at_page * a.c.heads + head) * a.c.page + in_page, sub, ok);
        }
    }
}

struct AppendLaunch {
    const KvqAppendArgs &a;
    hipStream_t s;
    template <int GT, int D, int BITS>
    void run() const {
        // at least 8 tokens of fewer than 2^26: at most 2^31 threads along x; at most 3 * 32767 heads, four
        // each: at most 24576 workgroups along y
        constexpr int64_t each = kAppendBlock / (D / 8);
        const int heads = a.q_heads + 2 * a.c.heads;
        const dim3 grid((unsigned)((a.tokens + each - 1) / each), (heads + kAppendHeads - 1) / kAppendHeads);
        hipLaunchKernelGGL((k_kvq_append<GT, D, BITS>), grid, dim3(kAppendBlock), 0, s, a);
    }
};

}  // namespace onebit

using namespace onebit;

extern "C" onebit_status_t kvq_append(const void *q, const void *k, const void *v, onebit_dtype_t dtype, int64_t tokens,
                                      int q_heads, int64_t q_token_stride, int64_t q_head_stride,
                                      int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                      int64_t v_head_stride, const int64_t *positions, const float *rotary,
                                      int64_t max_position, int rot_dim, int interleaved, const int64_t *slots,
                                      const kvq_cache_t *cache, void *q_out, int64_t out_token_stride,
                                      int64_t out_head_stride, void *stream) {
    KvqAppendArgs a{};
    const onebit_status_t st = kvq_check_rows(cache, dtype, tokens, &a.c);
    if (st != ONEBIT_OK) return st;
    if (q_heads < 0 || q_heads > 32767 || rot_dim < 16 || rot_dim > cache->head_dim || rot_dim % 16 || max_position < 1 ||
        max_position >= (int64_t{1} << 47) / rot_dim)
        return ONEBIT_ERR_INVALID;
    if (tokens == 0) return ONEBIT_OK;
    if (!k || !v || !slots || !positions || !rotary || (q_heads > 0 && (!q || !q_out))) return ONEBIT_ERR_INVALID;
    const int64_t unit = dtype == ONEBIT_F32 ? 4 : 8;  // elements in 16 bytes
    if (!aligned16(k) || !aligned16(v) || !aligned16(rotary) || !aligned_to(slots, 8) || !aligned_to(positions, 8) ||
        k_token_stride % unit || k_head_stride % unit || v_token_stride % unit || v_head_stride % unit)
        return ONEBIT_ERR_ALIGN;
    if (q_heads > 0 && (!aligned16(q) || !aligned16(q_out) || q_token_stride % unit || q_head_stride % unit ||
                        out_token_stride % unit || out_head_stride % unit))
        return ONEBIT_ERR_ALIGN;
    // rows of the result that would overlap
    const int dim = cache->head_dim;
    if (q_heads > 0 && ((tokens > 1 && out_token_stride > -dim && out_token_stride < dim) ||
                        (q_heads > 1 && out_head_stride > -dim && out_head_stride < dim)))
        return ONEBIT_ERR_INVALID;
    a.src[0] = q;
    a.src[1] = k;
    a.src[2] = v;
    a.token_stride[0] = q_token_stride;
    a.token_stride[1] = k_token_stride;
    a.token_stride[2] = v_token_stride;
    a.head_stride[0] = q_head_stride;
    a.head_stride[1] = k_head_stride;
    a.head_stride[2] = v_head_stride;
    a.out = q_out;
    a.out_token_stride = out_token_stride;
    a.out_head_stride = out_head_stride;
    a.positions = positions;
    a.slots = slots;
    a.rotary = rotary;
    a.max_position = max_position;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    kvq_dispatch(dtype, cache->head_dim, cache->bits, AppendLaunch{a, static_cast<hipStream_t>(stream)});
    return hip_status(hipGetLastError());
}
