// qsdp_linear.hip -- products of rows with a matrix kept in qsdp_quantize's codes, and the
// gradient of their input.
//   out_{t,o} = sum_i x_{t,i} w_{o,i},   dx_{t,i} = sum_o dy_{t,o} w_{o,i},   w = min_b + code * delta_b
#include "qsdp_linear.h"
#include "qsdp_rows.h"

namespace onebit {

// One weight, as qsdp_dequantize decodes it.
template <int BITS>
__device__ __forceinline__ float weight_at(const LinearArgs &a, int64_t i) {
    const int64_t b = i / a.bucket;
    const uint32_t c = BITS == 8 ? a.codes[i] : (a.codes[i >> 1] >> (4 * (i & 1))) & 15u;
    const float lo = a.lo[b], delta = __fdiv_rn(sub_rn(a.hi[b], lo), (float)((1 << BITS) - 1));
    return add_rn(lo, mul_rn((float)(int)c, delta));
}

// 32 x 32 results by 256 threads, binary32 throughout.
template <int GT, int BITS, bool GRAD>
__global__ __launch_bounds__(256) void k_qsdp_linear_plain(LinearArgs a) {
    __shared__ float xs[32][33], ws[32][33];
    const int64_t depth = GRAD ? a.rows : a.cols, width = GRAD ? a.cols : a.rows;
    const int64_t t0 = (int64_t)blockIdx.y * 32, o0 = (int64_t)blockIdx.x * 32;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t d0 = 0; d0 < depth; d0 += 32) {
        for (int r = ty; r < 32; r += 8) {
            const int64_t t = t0 + r, d = d0 + tx;
            xs[r][tx] = t < a.tokens && d < depth ? half_bits_to_float<GT>(a.x[t * a.x_stride + d]) : 0.0f;
            // linear: row o0 + r of the matrix, column d0 + tx; gradient: row d0 + r, column o0 + tx
            const int64_t row = (GRAD ? d0 : o0) + r, col = (GRAD ? o0 : d0) + tx;
            ws[r][tx] = row < a.rows && col < a.cols ? weight_at<BITS>(a, row * a.cols + col) : 0.0f;
        }
        __syncthreads();
        for (int d = 0; d < 32; ++d)
            for (int j = 0; j < 4; ++j)
                acc[j] = __fmaf_rn(xs[ty + 8 * j][d], GRAD ? ws[d][tx] : ws[tx][d], acc[j]);
        __syncthreads();
    }
    for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + ty + 8 * j, o = o0 + tx;
        if (t < a.tokens && o < width) a.out[t * a.out_stride + o] = (uint16_t)round_pair<GT>(acc[j], 0.0f);
    }
}

template <int GT, int BITS, int GROUPS, int NT, int MT, int WAVES, int SPLIT>
static void launch_rows(const LinearArgs &a, hipStream_t s) {
    constexpr int64_t each = 16 * NT * WAVES;
    hipLaunchKernelGGL((k_qsdp_rows<GT, BITS, GROUPS, NT, MT, WAVES, SPLIT>), dim3((unsigned)((a.rows + each - 1) / each)),
                       dim3(64 * WAVES * SPLIT), 0, s, a);
}
template <int GT, int BITS, int GROUPS>
static void launch_rows_tiles(const LinearArgs &a, hipStream_t s) {
    const bool wide = a.rows >= 64 * 256;
    if (a.tokens <= 16) {
        if (wide)
            a.cols >= 32 * kRowsChunk ? launch_rows<GT, BITS, GROUPS, 1, 1, 4, 2>(a, s) : launch_rows<GT, BITS, GROUPS, 1, 1, 4, 1>(a, s);
        else
            a.cols >= 32 * kRowsChunk ? launch_rows<GT, BITS, GROUPS, 1, 1, 1, 8>(a, s) : launch_rows<GT, BITS, GROUPS, 1, 1, 2, 4>(a, s);
    } else if (a.tokens <= 32) {
        wide ? launch_rows<GT, BITS, GROUPS, 2, 2, 4, 2>(a, s) : launch_rows<GT, BITS, GROUPS, 1, 2, 2, 4>(a, s);
    } else {
        wide ? launch_rows<GT, BITS, GROUPS, 2, 4, 4, 2>(a, s) : launch_rows<GT, BITS, GROUPS, 1, 4, 4, 2>(a, s);
    }
}
template <int GT, int BITS>
static void launch_rows_groups(const LinearArgs &a, hipStream_t s) {
    if (a.cols % kRowsChunk == 0 && a.bucket % kRowsChunk == 0)
        launch_rows_tiles<GT, BITS, 1>(a, s);
    else
        launch_rows_tiles<GT, BITS, 4>(a, s);
}

template <int GT, int BITS, bool GRAD>
static void launch(const LinearArgs &a, hipStream_t s) {
    if (!GRAD && a.tokens <= QSDP_LINEAR_EXACT_TOKENS) return launch_rows_groups<GT, BITS>(a, s);
    const int64_t width = GRAD ? a.cols : a.rows;
    // at most 65535 workgroups along y
    const int64_t most = 65535 * 32;
    for (int64_t t = 0; t < a.tokens; t += most) {
        LinearArgs x = a;
        x.x += t * a.x_stride;
        x.out += t * a.out_stride;
        x.tokens = a.tokens - t < most ? a.tokens - t : most;
        hipLaunchKernelGGL((k_qsdp_linear_plain<GT, BITS, GRAD>),
                           dim3((unsigned)((width + 31) / 32), (unsigned)((x.tokens + 31) / 32)), dim3(256), 0, s, x);
    }
}
template <bool GRAD>
static void dispatch(onebit_dtype_t dtype, int bits, const LinearArgs &a, hipStream_t s) {
    if (dtype == ONEBIT_BF16)
        bits == 4 ? launch<kGradBF16, 4, GRAD>(a, s) : launch<kGradBF16, 8, GRAD>(a, s);
    else
        bits == 4 ? launch<kGradF16, 4, GRAD>(a, s) : launch<kGradF16, 8, GRAD>(a, s);
}

constexpr int64_t kLinearMost = 1 << 24;  // tokens, rows and columns are below

static size_t linear_workspace(int64_t tokens, int64_t rows, int64_t cols) {
    if (tokens < 0 || tokens >= kLinearMost || rows < 1 || rows >= kLinearMost || cols < 32 || cols >= kLinearMost || cols % 32)
        return 0;
    return 16;
}

template <bool GRAD>
static onebit_status_t linear(const void *x, onebit_dtype_t dtype, int64_t tokens, int64_t x_stride,
                              const qsdp_matrix_t *w, void *out, int64_t out_stride, void *workspace,
                              size_t workspace_bytes, void *stream) {
    if (dtype == ONEBIT_F32) return ONEBIT_ERR_UNSUPPORTED;
    if (dtype != ONEBIT_BF16 && dtype != ONEBIT_F16) return ONEBIT_ERR_INVALID;
    if (!w || (w->bits != 4 && w->bits != 8) || w->bucket < 1 || w->bucket > 65536) return ONEBIT_ERR_INVALID;
    if (tokens < 0 || tokens >= kLinearMost || w->rows < 1 || w->rows >= kLinearMost || w->cols < 1 || w->cols >= kLinearMost)
        return ONEBIT_ERR_INVALID;
    if (w->cols % 32 || w->bucket % 32) return ONEBIT_ERR_UNSUPPORTED;
    if (tokens == 0) return ONEBIT_OK;
    const int64_t depth = GRAD ? w->rows : w->cols, width = GRAD ? w->cols : w->rows;
    if (!x || !out || !workspace || !w->codes || !w->bucket_min || !w->bucket_max) return ONEBIT_ERR_INVALID;
    if (tokens > 1 && (x_stride < depth || out_stride < width || x_stride >= int64_t{1} << 32 || out_stride >= int64_t{1} << 32))
        return ONEBIT_ERR_INVALID;
    if (workspace_bytes < linear_workspace(tokens, w->rows, w->cols)) return ONEBIT_ERR_INVALID;
    if (!aligned16(x) || (tokens > 1 && x_stride % 8) || !aligned_to(out, 2) || !aligned16(workspace) || !aligned16(w->codes) ||
        !aligned_to(w->bucket_min, 4) || !aligned_to(w->bucket_max, 4))
        return ONEBIT_ERR_ALIGN;
    LinearArgs a{};
    a.codes = w->codes;
    a.lo = w->bucket_min;
    a.hi = w->bucket_max;
    a.rows = w->rows;
    a.cols = w->cols;
    a.bucket = w->bucket;
    a.bucket_magic = (uint32_t)(((uint64_t{1} << 32) + w->bucket / 32 - 1) / (w->bucket / 32));
    a.x = static_cast<const uint16_t *>(x);
    a.x_stride = tokens > 1 ? x_stride : 0;
    a.out = static_cast<uint16_t *>(out);
    a.out_stride = tokens > 1 ? out_stride : 0;
    a.tokens = tokens;
    a.workspace = workspace;
    dispatch<GRAD>(dtype, w->bits, a, static_cast<hipStream_t>(stream));
    return hip_status(hipGetLastError());
}

}  // namespace onebit

using namespace onebit;

extern "C" size_t qsdp_linear_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols) {
    return linear_workspace(tokens, rows, cols);
}

extern "C" onebit_status_t qsdp_linear(const void *x, onebit_dtype_t dtype, int64_t tokens, int64_t x_stride,
                                       const qsdp_matrix_t *w, void *out, int64_t out_stride, void *workspace,
                                       size_t workspace_bytes, void *stream) {
    return linear<false>(x, dtype, tokens, x_stride, w, out, out_stride, workspace, workspace_bytes, stream);
}

extern "C" onebit_status_t qsdp_linear_grad(const void *dy, onebit_dtype_t dtype, int64_t tokens, int64_t dy_stride,
                                            const qsdp_matrix_t *w, void *dx, int64_t dx_stride, void *workspace,
                                            size_t workspace_bytes, void *stream) {
    return linear<true>(dy, dtype, tokens, dy_stride, w, dx, dx_stride, workspace, workspace_bytes, stream);
}
