// qsdp_linear.hip -- products of rows with a matrix kept in qsdp_quantize's codes, and the
// gradient of their input.
//   out_{t,o} = sum_i x_{t,i} w_{o,i},   dx_{t,i} = sum_o dy_{t,o} w_{o,i},   w = min_b + code * delta_b
#include <algorithm>

#include "qsdp_linear.h"
#include "qsdp_plan.h"
#include "qsdp_rows.h"
#include "qsdp_tile.h"

namespace onebit {

template <int GT, int BITS, int GROUPS, int NT, int MT, int WAVES, int SPLIT>
static void launch_rows(const LinearArgs &a, hipStream_t s) {
    constexpr int64_t each = 16 * NT * WAVES;
    hipLaunchKernelGGL((k_qsdp_rows<GT, BITS, GROUPS, NT, MT, WAVES, SPLIT>), dim3((unsigned)((a.rows + each - 1) / each)),
                       dim3(64 * WAVES * SPLIT), 0, s, a);
}
// The fewest rows of the matrix for a workgroup that leave one workgroup to a compute unit, the rest of its
// waves sharing the columns: 16, 32 or 64 (32 tokens, 4 bits: 8192 x 8192 38, 25, 32 us; 14336 x 4096 45,
// 27, 19).  Eight groups need more than four loads of columns.  Up to 128 rows a unit, 128 for more than 16 tokens
// (28672 x 8192 49 us against 64) and 64 otherwise (38 and 37); above, workgroups of a single group, of
// which more are on a unit at a time (32 tokens, 50304 x 1600 38 us against 47, one token 24 against 29).
template <int GT, int BITS, int GROUPS, int MT>
static void launch_rows_split(const LinearArgs &a, hipStream_t s) {
    const int64_t each = (a.rows + 255) / 256, loads = (a.cols * BITS + 8 * kRowsChunk - 1) / (8 * kRowsChunk);
    if (each <= 16 && loads > 4) return launch_rows<GT, BITS, GROUPS, 1, MT, 1, 8>(a, s);
    if (each <= 32) return launch_rows<GT, BITS, GROUPS, 1, MT, 2, 4>(a, s);
    if (each <= 64 || (each <= 128 && MT == 1)) return launch_rows<GT, BITS, GROUPS, 1, MT, 4, 2>(a, s);
    if constexpr (MT > 1)
        if (each <= 128) return launch_rows<GT, BITS, GROUPS, 2, MT, 4, 2>(a, s);
    launch_rows<GT, BITS, GROUPS, 1, MT, 4, 1>(a, s);
}
template <int GT, int BITS, int GROUPS>
static void launch_rows_tiles(const LinearArgs &a, hipStream_t s) {
    a.tokens <= 16 ? launch_rows_split<GT, BITS, GROUPS, 1>(a, s) : launch_rows_split<GT, BITS, GROUPS, 2>(a, s);
}

// Few tokens go to the streaming kernel: 32 over 28672 x 8192 49 us against the tiles' 84, over 8192 x 4096
// 15 to 16 against 24, over 4096 x 4096 14 against 18 (but 8 bits over 20000 x 1600 24 against 18).  With 33
// to 64 the tiles are ahead (16384 x 8192 52 us against 70, 8 bits over 28672 x 8192 102 against 129; 4 bits 89
// against 78).
static bool few_tokens(int64_t tokens) { return tokens <= QSDP_LINEAR_EXACT_TOKENS; }

template <int GT, int BITS>
static void launch_rows_groups(const LinearArgs &a, hipStream_t s) {
    // whether every step of a row has one bucket
    if (a.cols % kRowsChunk == 0 && a.bucket % kRowsChunk == 0)
        launch_rows_tiles<GT, BITS, 1>(a, s);
    else
        launch_rows_tiles<GT, BITS, 4>(a, s);
}

// Tiles, from the one that does most work a byte of LDS to the one that leaves fewest compute units
// idle.
using Tile0 = TileShape<256, 256, 128, 64, 1, 1>;
using Tile1 = TileShape<128, 128, 64, 64, 2, 2>;
using Tile2 = TileShape<64, 128, 32, 64, 2, 2>;
using Tile3 = TileShape<64, 64, 32, 64, 4, 2>;
template <class S>
constexpr bool is_planned(const PlannedShape &p) {
    return S::TM == p.tm && S::TN == p.tn && S::kGroups == p.groups;
}
static_assert(is_planned<Tile0>(kPlannedShapes[0]) && is_planned<Tile1>(kPlannedShapes[1]) &&
              is_planned<Tile2>(kPlannedShapes[2]) && is_planned<Tile3>(kPlannedShapes[3]), "the plan's shapes");

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
    if (!GRAD && few_tokens(l.tokens)) return launch_rows_groups<GT, BITS>(l, s);
    TileArgs a{};
    a.l = l;
    a.depth = GRAD ? l.rows : l.cols;
    a.width = GRAD ? l.cols : l.rows;
    const TilePlan p = tile_plan(l.tokens, a.width, a.depth, GRAD);
    a.tiles_m = (int32_t)p.tiles_m;
    a.tiles_n = (int32_t)p.tiles_n;
    a.splits = p.splits;
    a.steps = (int32_t)((a.depth + kTileDepth - 1) / kTileDepth);
    a.partial = static_cast<float *>(l.workspace);
    switch (p.shape) {
        case 0: return launch_tile<GT, BITS, GRAD, Tile0>(a, s);
        case 1: return launch_tile<GT, BITS, GRAD, Tile1>(a, s);
        case 2: return launch_tile<GT, BITS, GRAD, Tile2>(a, s);
        default: return launch_tile<GT, BITS, GRAD, Tile3>(a, s);
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

// Bytes that a call with a result of `width` columns uses at most; no fewer with more tokens.
static size_t linear_need(bool grad, int64_t tokens, int64_t width) {
    return !grad && few_tokens(tokens) ? 16 : (size_t)std::max(partial_room(tokens, width), int64_t{16});
}
static size_t linear_workspace(int64_t tokens, int64_t rows, int64_t cols) {
    if (tokens < 0 || tokens >= kLinearMost || rows < 1 || rows >= kLinearMost || cols < 32 || cols >= kLinearMost || cols % 32)
        return 0;
    return std::max(linear_need(false, tokens, rows), linear_need(true, tokens, cols));
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
    if (workspace_bytes < linear_need(GRAD, tokens, width)) return ONEBIT_ERR_INVALID;
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
