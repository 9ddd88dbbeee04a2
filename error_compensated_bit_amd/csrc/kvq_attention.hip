// kvq_attention.hip -- attention of new tokens over the coded key/value cache.
//   s_j = sm_scale * ks_j * <q, kc_j - z>,  out = sum_j softmax(s)_j * vs_j * (vc_j - z)
// with kc, vc the codes and ks, vs the scales of the attended rows.
#include <math.h>

#include <algorithm>

#include "kvq_step.h"

namespace onebit {

template <int GT, int D, int BITS>
__global__ __launch_bounds__(256) void k_kvq_attention(KvqAttnArgs a) {
    constexpr int V = D / 64;
    __shared__ float s_o[4][D];
    __shared__ float s_m[4], s_l[4];
    const int row = blockIdx.x, h = blockIdx.y, g = h / a.group;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // the last sequence that begins at or before the row
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (kvq_seq(a, mid).q0 <= row) lo = mid; else hi = mid;
    }
    const int b = lo;
    const KvqSeq seq = kvq_seq(a, b);
    if (row < seq.q0 || row >= seq.q0 + seq.len || (int64_t)seq.len * a.group <= a.max_rows) return;
    const int end = kvq_hi(seq, row - seq.q0), begin = kvq_lo(a, seq, row - seq.q0);
    float q[V], o[V], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        q[v] = half_bits_to_float<GT>(a.q[row * a.q_token_stride + h * a.q_head_stride + lane * V + v]);
        o[v] = 0.0f;
    }
    for (int j = begin + wave; j < end; j += 4) {
        const int64_t page = a.table[b * a.table_stride + (j >> a.c.shift)];
        if (page < 0 || page >= a.c.n_pages) continue;
        const int64_t r = (page * a.c.heads + g) * a.c.page + (j & (a.c.page - 1));
        float kc[V], vc[V], s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int d = lane * V + v;
            if (BITS == 8) {
                kc[v] = (float)a.c.codes[0][r * D + d];
                vc[v] = (float)a.c.codes[1][r * D + d];
            } else {
                kc[v] = (float)((a.c.codes[0][r * (D / 2) + (d >> 1)] >> (4 * (d & 1))) & 15);
                vc[v] = (float)((a.c.codes[1][r * (D / 2) + (d >> 1)] >> (4 * (d & 1))) & 15);
            }
            s = fmaf(q[v], kc[v] - (float)KvqLevels<BITS>::kZero, s);
        }
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1) s += __shfl_xor(s, x, 64);
        s *= a.c.scales[0][r] * a.scale2;
        if (a.q_sign) s = -s;
        if (a.cap2 > 0.0f) s = capped(s * a.cap_scale, a.cap2);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), e = exp2f(s - mn);
        const float w = e * a.c.scales[1][r];
        l = l * f + e;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(w, vc[v] - (float)KvqLevels<BITS>::kZero, o[v] * f);
        m = mn;
    }
    if (lane == 0) {
        s_m[wave] = m;
        s_l[wave] = l;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_o[wave][lane * V + v] = o[v];
    __syncthreads();
    if (wave) return;
    float mm = s_m[0];
    for (int w = 1; w < 4; ++w) mm = fmaxf(mm, s_m[w]);
    float ll = 0.0f;
    for (int w = 0; w < 4; ++w) ll += s_l[w] > 0.0f || s_l[w] != s_l[w] ? s_l[w] * exp2f(s_m[w] - mm) : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float t = 0.0f;
        for (int w = 0; w < 4; ++w)
            if (s_l[w] != 0.0f) t += s_o[w][lane * V + v] * exp2f(s_m[w] - mm);
        t = ll != 0.0f ? t / ll : 0.0f;
        const _Float16 th = (_Float16)t;
        a.out[((int64_t)row * a.q_heads + h) * D + lane * V + v] =
            GT == kGradBF16 ? (uint16_t)float_to_bf16_bits(t) : __builtin_bit_cast(uint16_t, th);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)row * a.q_heads + h] = ll != 0.0f ? (mm + log2f(ll)) * 0.693147180559945f : -INFINITY;
}

// Workgroups of a launch of the step kernel: three for each compute unit.
static int step_groups() {
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess) {
        int v = 0;
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0) cus = v;
    }
    return std::min(3 * cus, kStepMaxGroups);
}

static size_t attention_workspace(int64_t batch, int64_t total_q, int q_heads, int kv_heads, int head_dim) {
    if (batch < 0 || total_q < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || kv_heads > 32767) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    if (batch >= (1 << 26) || total_q > (0x7fffffff - 2048) / q_heads) return 0;
    const size_t rows = head_dim == 256 ? 16 : 32;
    return kStepHeader + (size_t)step_groups() * 2 * rows * (head_dim + 2) * sizeof(float);
}

template <int GT, int D, int BITS>
static void launch(KvqAttnArgs a, hipStream_t s) {
    constexpr int kWide = D == 256 ? 1 : 2;
    a.max_rows = 32;
    if (a.q_offsets || (int64_t)a.q_uniform * a.group > a.max_rows)
        hipLaunchKernelGGL((k_kvq_attention<GT, D, BITS>), dim3(a.total_q, a.q_heads), dim3(256), 0, s, a);
    if (!a.q_offsets && (int64_t)a.q_uniform * a.group > a.max_rows) return;
    const bool wide = kWide == 2 && (a.group > 16 || (!a.q_offsets && a.q_uniform * a.group > 16));
    const unsigned groups = (unsigned)step_groups();
    const int batch = a.batch;
    for (int b = 0; b < batch; b += kStepSeqs) {
        KvqAttnArgs x = a;
        x.batch = std::min(batch - b, kStepSeqs);
        if (a.q_offsets) x.q_offsets = a.q_offsets + b;
        x.kv_lens = a.kv_lens + b;
        x.table = a.table + b * a.table_stride;
        x.q_first = b * a.q_uniform;
        if (wide)
            hipLaunchKernelGGL((k_kvq_step<GT, D, BITS, kWide>), dim3(groups), dim3(kStepBlock), 0, s, x);
        else
            hipLaunchKernelGGL((k_kvq_step<GT, D, BITS, 1>), dim3(groups), dim3(kStepBlock), 0, s, x);
    }
}

template <int GT, int D>
static void launch_bits(int bits, const KvqAttnArgs &a, hipStream_t s) {
    if (bits == 4)
        launch<GT, D, 4>(a, s);
    else
        launch<GT, D, 8>(a, s);
}
template <int GT>
static void launch_dim(int dim, int bits, const KvqAttnArgs &a, hipStream_t s) {
    if (dim == 64)
        launch_bits<GT, 64>(bits, a, s);
    else if (dim == 128)
        launch_bits<GT, 128>(bits, a, s);
    else
        launch_bits<GT, 256>(bits, a, s);
}

}  // namespace onebit

using namespace onebit;

extern "C" size_t kvq_attention_workspace_bytes(int64_t batch, int64_t total_q, int q_heads, int kv_heads,
                                                int head_dim) {
    return attention_workspace(batch, total_q, q_heads, kv_heads, head_dim);
}

extern "C" onebit_status_t kvq_attention(const void *q, onebit_dtype_t dtype, int64_t total_q, int q_heads,
                                         int64_t q_token_stride, int64_t q_head_stride, const int32_t *q_offsets,
                                         const int32_t *kv_lens, int64_t batch, const int32_t *block_table,
                                         int64_t max_pages, int64_t table_stride, const kvq_cache_t *cache,
                                         double sm_scale, double softcap, int window, void *out, float *lse,
                                         void *workspace, size_t workspace_bytes, void *stream) {
    KvqAttnArgs a{};
    if (dtype == ONEBIT_F32) return ONEBIT_ERR_UNSUPPORTED;
    if (dtype != ONEBIT_BF16 && dtype != ONEBIT_F16) return ONEBIT_ERR_INVALID;
    const onebit_status_t st = kvq_check_cache(cache, &a.c);
    if (st != ONEBIT_OK) return st;
    const size_t need = attention_workspace(batch, total_q, q_heads, cache->kv_heads, cache->head_dim);
    if (need == 0) return ONEBIT_ERR_INVALID;
    if (max_pages < 0 || max_pages > (0x7fffffff - 2048) / cache->page || (batch > 1 && table_stride < max_pages))
        return ONEBIT_ERR_INVALID;
    if (window < 0 || !(softcap >= 0.0) || !__builtin_isfinite((float)softcap) || !__builtin_isfinite((float)sm_scale))
        return ONEBIT_ERR_INVALID;
    if (batch == 0 || total_q == 0) return ONEBIT_OK;
    if (!q_offsets && total_q % batch) return ONEBIT_ERR_INVALID;
    if (!q || !kv_lens || !out || !workspace || (max_pages > 0 && !block_table)) return ONEBIT_ERR_INVALID;
    if (workspace_bytes < need) return ONEBIT_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || q_token_stride % 8 || q_head_stride % 8 ||
        !aligned_to(kv_lens, 4) || !aligned_to(block_table, 4) || !aligned_to(q_offsets, 4) || !aligned_to(lse, 4))
        return ONEBIT_ERR_ALIGN;
    a.q = static_cast<const uint16_t *>(q);
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.q_offsets = q_offsets;
    a.kv_lens = kv_lens;
    a.table = block_table;
    a.table_stride = table_stride;
    a.batch = (int32_t)batch;
    a.total_q = (int32_t)total_q;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    // without pages there is nothing to read, whatever the table says
    a.max_tokens = a.c.n_pages ? (int32_t)(max_pages * cache->page) : 0;
    a.q_uniform = q_offsets ? 0 : (int32_t)(total_q / batch);
    a.window = window;
    a.scale2 = (float)(__builtin_fabs(sm_scale) * 1.4426950408889634);
    a.q_sign = sm_scale < 0.0 ? 0x80000000u : 0u;
    a.cap2 = (float)(softcap * 1.4426950408889634);
    a.cap_scale = softcap > 0.0 ? (float)(2.0 / softcap) : 0.0f;
    a.workspace = workspace;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == ONEBIT_BF16)
        launch_dim<kGradBF16>(cache->head_dim, cache->bits, a, s);
    else
        launch_dim<kGradF16>(cache->head_dim, cache->bits, a, s);
    return hip_status(hipGetLastError());
}
