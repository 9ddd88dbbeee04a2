// qsdp_linear.hip -- products of rows with a matrix kept in qsdp_quantize's codes, and the
// gradient of their input.
//   out_{t,o} = sum_i x_{t,i} w_{o,i},   dx_{t,i} = sum_o dy_{t,o} w_{o,i},   w = min_b + code * delta_b
#include <algorithm>

#include "qsdp_linear.h"
#include "qsdp_rows.h"
#include "qsdp_tile.h"

namespace onebit {

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

using BigTile = TileShape<256, 256, 128, 64, 1, 1>;
using SmallTile = TileShape<128, 128, 64, 64, 2, 2>;

// How a product is cut up: its tiles and how many workgroups share the depth of each.
struct TilePlan {
    bool big;
    int64_t tiles_m, tiles_n;
    int splits;
    size_t bytes;  // of partial results
};
static TilePlan tile_plan(int64_t tokens, int64_t width, int64_t depth) {
    TilePlan p;
    const int64_t big = ((tokens + 255) / 256) * ((width + 255) / 256);
    p.big = big >= 192;
    const int64_t side = p.big ? 256 : 128, room = 256, steps = (depth + kTileDepth - 1) / kTileDepth;
    p.tiles_m = (tokens + side - 1) / side;
    p.tiles_n = (width + side - 1) / side;
    const int64_t tiles = p.tiles_m * p.tiles_n;
    p.splits = (int)std::max<int64_t>(1, std::min({room / tiles, steps / 4, (int64_t)64}));
    p.bytes = p.splits > 1 ? (size_t)tiles * p.splits * side * side * sizeof(float) : 0;
    return p;
}

template <int GT, int BITS, bool GRAD, class S>
static void launch_tile(const TileArgs &a, hipStream_t s) {
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    hipLaunchKernelGGL((k_qsdp_tile<GT, BITS, GRAD, S>), dim3((unsigned)(tiles * a.splits)), dim3(S::kThreads * S::kGroups), 0, s, a);
    if (a.splits > 1)
        hipLaunchKernelGGL((k_qsdp_tile_join<GT, S>), dim3((unsigned)((tiles * S::kWaves * S::kFrags + 3) / 4)), dim3(256), 0,
                           s, a);
}

template <int GT, int BITS, bool GRAD>
static void launch(const LinearArgs &l, hipStream_t s) {
    if (!GRAD && l.tokens <= QSDP_LINEAR_EXACT_TOKENS) return launch_rows_groups<GT, BITS>(l, s);
    TileArgs a{};
    a.l = l;
    a.depth = GRAD ? l.rows : l.cols;
    a.width = GRAD ? l.cols : l.rows;
    const TilePlan p = tile_plan(l.tokens, a.width, a.depth);
    a.tiles_m = (int32_t)p.tiles_m;
    a.tiles_n = (int32_t)p.tiles_n;
    a.splits = p.splits;
    a.steps = (int32_t)((a.depth + kTileDepth - 1) / kTileDepth);
    a.partial = static_cast<float *>(l.workspace);
    p.big ? launch_tile<GT, BITS, GRAD, BigTile>(a, s) : launch_tile<GT, BITS, GRAD, SmallTile>(a, s);
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
    if (tokens == 0) return 16;
    const size_t linear = tokens > QSDP_LINEAR_EXACT_TOKENS ? tile_plan(tokens, rows, cols).bytes : 0;
    return std::max({(size_t)16, linear, tile_plan(tokens, cols, rows).bytes});
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
    if (tokens > 1 && (x_stride < depth || out_stride < width || x_stride >= int64_t{1} << 23 || out_stride >= int64_t{1} << 32))
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
