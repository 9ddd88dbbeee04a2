// kvq_attention.hip -- attention of new tokens over the coded key/value cache.
//   s_j = sm_scale * ks_j * <q, kc_j - z>,  out = sum_j softmax(s)_j * vs_j * (vc_j - z)
// with kc, vc the codes and ks, vs the scales of the attended rows.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "kvq_chunk.h"
#include "kvq_step.h"

namespace onebit {

// Compute units of the current device, asked for once for each device.
static int compute_units() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int cus = known[dev].load(std::memory_order_relaxed);
    if (cus == 0) {
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
        known[dev].store(cus, std::memory_order_relaxed);
    }
    return cus;
}

// Workgroups of a launch: as many as are resident at once.
static int step_groups() { return std::min(3 * compute_units(), kStepMaxGroups); }
static int chunk_groups() { return std::min(compute_units(), kChunkMaxGroups); }
// Waves of a chunk workgroup.  With 256 dimensions a wave's outputs, queries and scores
// need more than half of a SIMD's registers, so there is room for one on each.
constexpr int chunk_waves(int dim) { return dim == 256 ? 4 : 8; }

// The step kernel's counters, then the partial results of either kernel (one runs after
// the other).
static size_t step_bytes(int dim) {
    return (size_t)step_groups() * 2 * (dim == 128 ? 32 : 16) * (dim + 2) * sizeof(float);
}
static size_t chunk_bytes(int dim) {
    return kChunkMaxGroups * sizeof(ChunkSplit) +
           (size_t)chunk_groups() * 2 * chunk_waves(dim) * 32 * (dim + 2) * sizeof(float);
}

static size_t attention_workspace(int64_t batch, int64_t total_q, int q_heads, int kv_heads, int head_dim) {
    if (batch < 0 || total_q < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || kv_heads > 32767) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    if (batch >= (1 << 26) || total_q > (0x7fffffff - 2048) / q_heads) return 0;
    return kStepHeader + std::max(step_bytes(head_dim), chunk_bytes(head_dim));
}

// The sequences [b, b + count) of a call, as a launch's own.
static KvqAttnArgs slice(const KvqAttnArgs &a, int b, int count) {
    KvqAttnArgs x = a;
    x.batch = std::min(a.batch - b, count);
    if (a.q_offsets) x.q_offsets = a.q_offsets + b;
    x.kv_lens = a.kv_lens + b;
    x.table = a.table + b * a.table_stride;
    x.q_first = b * a.q_uniform;
    return x;
}

template <int GT, int D, int BITS>
static void launch(KvqAttnArgs a, hipStream_t s) {
    constexpr int kWide = D == 128 ? 2 : 1, kWaves = chunk_waves(D);
    // Measured with 48 rows against the chunk kernel (us, 8 x 4096 tokens / 32 x 16384, 8 heads):
    // bf16 heads of 64 25 : 42 / 214 : 298, of 128 38 : 55 / 374 : 444, fp16 39 : 70 / 390 : 587; one
    // sequence of 16384 38 : 37; with 64 rows and bf16 57 : 55 / 623 : 444.
    a.max_rows = 48;
    const int64_t rows = (int64_t)a.q_uniform * a.group;  // of every sequence, where that is known
    if (a.q_offsets || rows <= a.max_rows) {
        // 17 to 32 rows at once read the cache once, but leave room for fewer workgroups and join more
        // slowly.  That pays with heads of 128, where a second reading would come from memory and not
        // from the 256 MB cache in front of it (as far as the tables tell): 32 rows, 8 heads, 32 x 16384
        // tokens 270 : 329 us, but 32 x 2000 63 : 58, 8 x 4096 60 : 39, 1 x 16384 102 : 48.  With heads
        // of 64 it is 180 : 181 at the best.
        const int64_t most = a.q_offsets ? a.group : rows;
        const bool wide = kWide == 2 && most > 16 && most <= 32 &&
                          (double)a.batch * a.c.heads * a.max_tokens * (D * BITS / 4 + 8) > 0x1p28;
        for (int b = 0; b < a.batch; b += kStepSeqs) {
            const KvqAttnArgs x = slice(a, b, kStepSeqs);
            if (wide)
                hipLaunchKernelGGL((k_kvq_step<GT, D, BITS, kWide>), dim3(step_groups()), dim3(kStepBlock), 0, s, x);
            else
                hipLaunchKernelGGL((k_kvq_step<GT, D, BITS, 1>), dim3(step_groups()), dim3(kStepBlock), 0, s, x);
        }
    }
    // without offsets that say otherwise, no sequence has more than all the rows
    if (a.q_offsets ? (int64_t)a.total_q * a.group > a.max_rows : rows > a.max_rows) {
        for (int b = 0; b < a.batch; b += kChunkSeqs) {
            KvqAttnArgs x = slice(a, b, kChunkSeqs);
            x.workspace = static_cast<char *>(a.workspace) + kStepHeader;
            hipLaunchKernelGGL((k_kvq_chunk<GT, D, BITS, kWaves>), dim3(chunk_groups()), dim3(64 * kWaves), 0, s, x);
            hipLaunchKernelGGL((k_kvq_chunk_join<GT, D, kWaves>), dim3(8 * compute_units()), dim3(64 * kJoinWaves), 0, s, x,
                               chunk_groups());
        }
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
    // (what the kernels make of both stays far from fp32's ends)
    if (window < 0 || !(softcap == 0.0 || (softcap >= 0x1p-64 && softcap <= 0x1p64)) || !(__builtin_fabs(sm_scale) <= 0x1p64))
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
