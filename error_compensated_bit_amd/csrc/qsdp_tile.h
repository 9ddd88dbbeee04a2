// qsdp_tile.h -- many rows times a coded matrix or its transpose: bound by the matrix cores.
//   linear:    out_{t,o} = sum_d x_{t,d} w_{o,d}       (o a row of the matrix, d a column)
//   gradient:  out_{t,o} = sum_d x_{t,d} w_{d,o}       (o a column, d a row)
// A workgroup has TM x TN results and goes through the depth in steps of 64.  A step's x
// and its weights, expanded once for all TM rows and rounded to x's type, lie in LDS twice over:
// while one is multiplied the next is written and the one after that is on its way from memory.
// The matrix cores take both operands in one type, so a weight is rounded to 8 or 11 bits: a second
// product with what the rounding leaves would double the products (floor of 2048 x 16384 x 4096: 200 us,
// then 400) and the weights' half of LDS, which the first shape does not have.  What that costs, against
// 64 bits in root mean square: 0.0023 instead of the result's own 0.0017 in bf16, 0.00029 instead of
// 0.00021 in fp16.
// Each wave writes first and multiplies then: of two waves on a SIMD one comes to its products
// while the other still expands (half of them the other way round: twice the code, and no faster).
//
// LDS: rows of 64 values (128 bytes) of x and of weights, the 16-byte pieces of row r in the order
// p ^ x_swizzle(r) or p ^ w_swizzle(r), so that what eight lanes read or write at once lies in
// different banks, while rows a multiple of 32 apart (of 16, for x) have one order: their
// addresses differ by a constant.  An operand of v_mfma_f32_16x16x32 is one piece of 16 rows.  Weights are the first
// operand, so that a lane holds four neighbouring results of one row of x.
//
// Measured: 2048 x 16384 x 4096, 4 bits, bf16, 260 to 290 us (0.95 to 1.06 PFLOP/s; the library's product
// with decoded weights, 179 to 200); gradient of 4096 x 1600 x 6400 120 to 126 us (87 to 97), of 500 x 1600 x
// 50257, fp16, 8 bits, 120 to 132 us (270).  In the first the matrix cores are busy in 44% of the compute
// units' time, LDS in 44% and in 17% for bank conflicts; in the gradients 42%, 48% and 16%.
// Small products are bound by a step's chain of waits, 1.2 us: 333 x 4800 x 1600 17 us, 77 x 4096 x 4096
// 18 to 20 (matrix cores 15%).
#pragma once

#include "qsdp_linear.h"
#include "qsdp_plan.h"

namespace onebit {

// TM x TN results of a workgroup, WM x WN of a wave; GROUPS of waves share the depth, each with
// buffers of its own; AHEAD steps of a group are on their way from memory.
template <int TM_, int TN_, int WM_, int WN_, int GROUPS, int AHEAD>
struct TileShape {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, kGroups = GROUPS, kAhead = AHEAD;
    // of a group
    static constexpr int kWaves = (TM / WM) * (TN / WN), kThreads = 64 * kWaves;
    static constexpr int kXPieces = TM * 8 / kThreads;  // of a thread
    static constexpr int kFrags = (WM / 16) * (WN / 16);
    static constexpr int kOccupancy = kWaves * GROUPS / 4;  // waves on a SIMD
    static_assert(kThreads == 2 * TN, "a thread expands 32 codes of a step");
};

struct TileArgs {
    LinearArgs l;
    int64_t depth, width;
    int32_t tiles_m, tiles_n;
    int32_t splits;      // workgroups that share the depth of a tile
    int32_t steps;       // of the whole depth
    float *partial;      // [tile][split][wave][frag][lane][4] where splits > 1
};

__device__ __forceinline__ int x_swizzle(int r) { return (r ^ ((r >> 3) & 1)) & 7; }
__device__ __forceinline__ int w_swizzle(int r) { return (r ^ ((r >> 3) & 3)) & 7; }

// Two weights of one row, rounded once more to x's type.
template <int GT>
__device__ __forceinline__ uint32_t weight_pair(float c0, float c1, float delta, float lo) {
    return round_pair<GT>(__fmaf_rn(c0, delta, lo), __fmaf_rn(c1, delta, lo));
}

// Four neighbouring results of row t, as far as they are in it.
template <int GT>
__device__ __forceinline__ void store_results(const TileArgs &a, int64_t t, int64_t o, f32x4_v v) {
    if (t >= a.l.tokens || o >= a.width) return;
    uint16_t *p = a.l.out + t * a.l.out_stride + o;
    const uint32_t w[2] = {round_pair<GT>(v[0], v[1]), round_pair<GT>(v[2], v[3])};
    if (o + 4 <= a.width && ((uintptr_t)p & 7) == 0) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (o + e < a.width) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

template <int GT, int BITS, bool GRAD, class S>
__global__ __launch_bounds__(S::kThreads * S::kGroups, S::kOccupancy) void k_qsdp_tile(TileArgs a) {
    constexpr int kXBytes = S::TM * 128, kWBytes = S::TN * 128;
    constexpr int kScaleBytes = GRAD ? S::kThreads * 8 : 0;
    constexpr int kGroupBytes = 2 * (kXBytes + kWBytes + kScaleBytes);
    __shared__ __attribute__((aligned(16))) char s_all[S::kGroups * kGroupBytes];
    const int group = S::kGroups == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / S::kThreads);
    char *s_mem = s_all + group * kGroupBytes;
    const int tid = threadIdx.x - group * S::kThreads, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;

    // ---- which tile, which part of the depth.  Workgroups go round the XCDs: each XCD takes consecutive ones.
    int at = blockIdx.x;
    {
        const int total = gridDim.x, per = total >> 3, more = total & 7, xcd = at & 7;
        at = (at >> 3) + xcd * per + min(xcd, more);
    }
    const int split = at % a.splits, tile = at / a.splits;
    const int tm = tile % a.tiles_m, tn = tile / a.tiles_m;
    const int64_t t0 = (int64_t)tm * S::TM, o0 = (int64_t)tn * S::TN;
    // this group's steps; every group of the workgroup goes through as many
    const int first = (int)((int64_t)a.steps * split / a.splits), behind = (int)((int64_t)a.steps * (split + 1) / a.splits);
    const int each = (behind - first + S::kGroups - 1) / S::kGroups;
    const int begin = min(first + group * each, behind), end = min(begin + each, behind);
    const int whole = (int)(a.depth / kTileDepth);  // steps that are full

    const auto first_of = [&](int64_t base, int64_t count, int r) { return (uint32_t)(min(base + r, count - 1) - base); };

    // ---- x: rows (tid >> 3) + kThreads / 8 * m, piece tid & 7; by offsets from the tile's first row, which
    // fit 32 bits (256 rows, strides below 2^23)
    const char *x = reinterpret_cast<const char *>(a.l.x + t0 * a.l.x_stride);
    uint32_t x_off[S::kXPieces];
#pragma unroll
    for (int m = 0; m < S::kXPieces; ++m)
        x_off[m] = first_of(t0, a.l.tokens, (tid >> 3) + S::kThreads / 8 * m) * (2 * (uint32_t)a.l.x_stride) + 16 * (tid & 7);
    constexpr int kA = S::kAhead;
    u32x4_v xr[kA][S::kXPieces];

    // ---- codes
    const uint32_t row_parts = (uint32_t)(a.l.cols >> 5), bucket_parts = (uint32_t)a.l.bucket >> 5;
    const uint32_t row_bytes = row_parts * (4 * BITS);
    constexpr int kCodeWords = GRAD ? 8 : BITS;  // columns of eight rows, or words of 32 codes
    uint32_t code[kA][kCodeWords];
    float lo[kA + 2], hi[kA + 2];  // (two more for the gradient's first tables)
    // linear: this thread's row and half of a step.  gradient: rows 8 (tid / (TN / 4)) + 0 .. 7 of a step, columns
    // 4 (tid % (TN / 4)) + 0 .. 3, and an entry of the step's table of minima and steps: row tid / (TN / 32),
    // columns 32 (tid % (TN / 32)) + 0 .. 31.
    const int c_row = GRAD ? 8 * (tid / (S::TN / 4)) : tid >> 1, c_col = GRAD ? 4 * (tid % (S::TN / 4)) : 32 * (tid & 1);
    const int e_row = tid / (S::TN / 32), e_part = tid % (S::TN / 32);
    const uint8_t *codes = a.l.codes;
    const float *los = a.l.lo, *his = a.l.hi;
    uint32_t code_off, part, step_parts = 0;  // part: in front of the thread's next part in its bucket
    int64_t bucket = 0, step_buckets = 0;
    if (GRAD) {
        codes += o0 * BITS >> 3;
        code_off = (uint32_t)c_row * row_bytes + (first_of(o0 >> 2, a.l.cols >> 2, c_col >> 2) * BITS >> 1);
        const int64_t p = (int64_t)begin * kTileDepth + e_row;
        const Bucket b = bucket_of(p * row_parts + min((uint32_t)(o0 >> 5) + e_part, row_parts - 1), bucket_parts);
        bucket = b.index;
        part = b.part;
        const Bucket d = bucket_of((int64_t)kTileDepth * row_parts, bucket_parts);
        step_buckets = d.index;
        step_parts = d.part;
    } else {
        const uint32_t r = first_of(o0, a.l.rows, c_row);
        const Bucket b = bucket_of(o0 * row_parts, bucket_parts);
        codes += o0 * row_bytes;
        los += b.index;
        his += b.index;
        code_off = r * row_bytes;
        const uint32_t parts = b.part + r * row_parts;
        bucket = parts / bucket_parts;
        part = parts - (uint32_t)bucket * bucket_parts;
    }

    // minima and maxima of step s (gradient: to be called for every step in turn)
    const auto load_scales = [&](int s, int slot) {
        if (GRAD) {
            const bool in = s < end && (int64_t)s * kTileDepth + e_row < a.l.rows;
            const int64_t b = in ? bucket : 0;
            lo[slot] = los[b];
            hi[slot] = his[b];
            if (!in) lo[slot] = hi[slot] = 0.0f;  // behind the last row: weights of 0
            bucket += step_buckets;
            part += step_parts;
            if (part >= bucket_parts) {
                part -= bucket_parts;
                ++bucket;
            }
        } else {
            const uint32_t c = (uint32_t)s * 2 + (tid & 1), k = part + min(c, row_parts - 1);
            const uint32_t b = (uint32_t)bucket + (bucket_parts == 1 ? k : __umulhi(k, a.l.bucket_magic));
            lo[slot] = los[b];
            hi[slot] = his[b];
            if (c >= row_parts) lo[slot] = hi[slot] = 0.0f;  // behind the row's end: weights of 0
        }
    };
    // (steps behind the last are the last one again, not used: a branch around the loads would make the
    // compiler wait for all that are under way)
    const auto load = [&](int step, int slot) {
        const int s = max(min(step, end - 1), first);
        const int64_t d0 = (int64_t)s * kTileDepth;
        if (!GRAD) load_scales(s, slot);
        if (s < whole) {
#pragma unroll
            for (int m = 0; m < S::kXPieces; ++m)
                xr[slot][m] = *reinterpret_cast<const u32x4_v *>(x + 2 * d0 + x_off[m]);
        } else {
            // the depth's end: value by value, the last one and zeros for those behind it
            const int left = (int)(a.depth - d0) - 8 * (tid & 7);
#pragma unroll
            for (int m = 0; m < S::kXPieces; ++m) {
                const uint16_t *p = reinterpret_cast<const uint16_t *>(x + 2 * d0 + x_off[m]);
                uint32_t v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = p[min(k, left - 1)];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = k < left ? v[k] : 0u;
                xr[slot][m] = (u32x4_v){v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
            }
        }
        if (GRAD) {
            const uint8_t *p = codes + d0 * row_bytes;
            const auto code_at = [&](const uint8_t *q) -> uint32_t {
                return BITS == 4 ? *reinterpret_cast<const uint16_t *>(q) : *reinterpret_cast<const uint32_t *>(q);
            };
            if (s < whole) {
#pragma unroll
                for (int r = 0; r < 8; ++r) code[slot][r] = code_at(p + (uint64_t)r * row_bytes + code_off);
            } else {
                // (behind the last row: the last one, times the table's zeros)
                const int last = (int)(a.l.rows - d0) - 1;
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    code[slot][r] = code_at(p + (code_off - (uint32_t)(c_row - min(c_row + r, last)) * row_bytes));
            }
        } else {
            const uint32_t off = code_off + (min((uint32_t)s * kTileDepth + c_col, row_parts * 32 - 32) * BITS >> 3);
#pragma unroll
            for (int k = 0; k < BITS / 4; ++k) {
                const uint4 v = *reinterpret_cast<const uint4 *>(codes + off + 16 * k);
                code[slot][4 * k] = v.x;
                code[slot][4 * k + 1] = v.y;
                code[slot][4 * k + 2] = v.z;
                code[slot][4 * k + 3] = v.w;
            }
        }
    };

    const auto x_at = [&](int buffer) { return reinterpret_cast<u32x4_v *>(s_mem + buffer * kXBytes); };
    const auto w_at = [&](int buffer) { return reinterpret_cast<u32x4_v *>(s_mem + 2 * kXBytes + buffer * kWBytes); };
    const auto table_at = [&](int buffer) {
        return reinterpret_cast<float2 *>(s_mem + 2 * (kXBytes + kWBytes) + buffer * kScaleBytes);
    };
    const auto keep_table = [&](int buffer, int slot) {
        table_at(buffer)[tid] = make_float2(lo[slot], bucket_delta<BITS>(lo[slot], hi[slot]));
    };
    const auto byte_of = [](uint32_t w, int k) -> float { return (float)((w >> (8 * k)) & 255u); };

    // x and weights of the step in `slot` into `buffer`
    const auto store = [&](int buffer, int slot) {
        u32x4_v *xs = x_at(buffer) + 8 * (tid >> 3) + ((tid & 7) ^ x_swizzle(tid >> 3)), *ws = w_at(buffer);
#pragma unroll
        for (int m = 0; m < S::kXPieces; ++m) xs[S::kThreads * m] = xr[slot][m];
        if (GRAD) {
            // the minima and steps of two rows at a time, for all four columns
            const float2 *e = table_at(buffer) + c_row * (S::TN / 32) + (c_col >> 5);
            u32x4_v v[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2 e0 = e[2 * p * (S::TN / 32)], e1 = e[(2 * p + 1) * (S::TN / 32)];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t c0 = code[slot][2 * p] >> (BITS * k), c1 = code[slot][2 * p + 1] >> (BITS * k);
                    constexpr uint32_t m = (1u << BITS) - 1;
                    v[k][p] = round_pair<GT>(__fmaf_rn((float)(c0 & m), e0.y, e0.x), __fmaf_rn((float)(c1 & m), e1.y, e1.x));
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int o = c_col + k;
                ws[8 * o + ((c_row >> 3) ^ w_swizzle(o))] = v[k];
            }
        } else {
            const float delta = bucket_delta<BITS>(lo[slot], hi[slot]);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                u32x4_v v;
                if (BITS == 4) {
                    const uint32_t even = code[slot][p] & 0x0f0f0f0fu, odd = (code[slot][p] >> 4) & 0x0f0f0f0fu;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = weight_pair<GT>(byte_of(even, k), byte_of(odd, k), delta, lo[slot]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t c = code[slot][(2 * p + (k >> 1)) % kCodeWords];
                        v[k] = weight_pair<GT>(byte_of(c, 2 * (k & 1)), byte_of(c, 2 * (k & 1) + 1), delta, lo[slot]);
                    }
                }
                ws[8 * c_row + ((4 * (tid & 1) + p) ^ w_swizzle(c_row))] = v;
            }
        }
    };

    // ---- products: this wave's part of the tile
    constexpr int kM = S::WM / 16, kN = S::WN / 16;
    const int wm = (wave % (S::TM / S::WM)) * S::WM, wn = (wave / (S::TM / S::WM)) * S::WN;
    f32x4_v acc[kN][kM];
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < kM; ++j) acc[i][j] = (f32x4_v){0.0f, 0.0f, 0.0f, 0.0f};
    // piece 4 k + g of row n of a tile of 16; odd tiles of weights have another order
    const int x_first = 8 * (wm + n), w_first = 8 * (wn + n);
    int x_piece[2], w_piece[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        x_piece[k] = x_first + ((4 * k + g) ^ x_swizzle(n));
#pragma unroll
        for (int i = 0; i < 2; ++i) w_piece[k][i] = w_first + ((4 * k + g) ^ w_swizzle(n + 16 * i));
    }
    const auto multiply = [&](int buffer) {
        const u32x4_v *xs = x_at(buffer), *ws = w_at(buffer);
#pragma unroll
        for (int k = 0; k < kTileDepth / 32; ++k) {
            u32x4_v wf[kN], xf[kM];
#pragma unroll
            for (int i = 0; i < kN; ++i) wf[i] = ws[w_piece[k][i & 1] + 128 * i];
#pragma unroll
            for (int j = 0; j < kM; ++j) xf[j] = xs[x_piece[k] + 128 * j];
            // (the order that leaves the compiler the better schedule: 285 against 289 us, 130 against 145)
#pragma unroll
            for (int q = 0; q < kN * kM; ++q) {
                const int i = GRAD ? q % kN : q / kM, j = GRAD ? q / kN : q % kM;
                acc[i][j] = product16<GT>(wf[i], xf[j], acc[i][j]);
            }
        }
    };

    // ---- the pipeline.  Step begin + i goes through slot i % kA and buffer i % 2.
    static_assert(kA <= 2, "steps of the loop's body");
    // Everything is asked for before the first wait.
    if (GRAD) {
        load_scales(begin, kA);
        load_scales(begin + 1, kA + 1);
    }
#pragma unroll
    for (int i = 0; i < kA; ++i) load(begin + i, i);
    if (GRAD) {
#pragma unroll
        for (int i = 0; i < kA; ++i) load_scales(begin + 2 + i, i);
        keep_table(0, kA);
        keep_table(1, kA + 1);
        __syncthreads();
    }
    store(0, 0);
    load(begin + kA, 0);
    __syncthreads();
    // the step after s (= begin + u, for what u decides) into LDS, another one on its way
    const auto advance = [&](int s, int u) {
        store((u + 1) & 1, (u + 1) % kA);
        if (GRAD) {
            keep_table(u & 1, u % kA);
            load_scales(s + 2 + kA, u % kA);
        }
        load(s + 1 + kA, (u + 1) % kA);
    };
    for (int i = 0; i < each; i += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (i + u >= each) break;
            advance(begin + i + u, u);
            // (The condition holds without groups, but without the branch the compiler mixes the linear
            // product's expansion into its products: 305 us for 289.  The gradient gains by it, 130 for 135.)
            if ((GRAD && S::kGroups == 1) || begin + i + u < end) multiply(u);
            __syncthreads();
        }
    }

    // ---- the groups' sums, in their order
    if (S::kGroups > 1) {
        f32x4_v *s_sum = reinterpret_cast<f32x4_v *>(s_all);
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
#pragma unroll
                for (int j = 0; j < kM; ++j)
                    s_sum[(((group - 1) * S::kWaves + wave) * S::kFrags + i * kM + j) * 64 + lane] = acc[i][j];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int k = 0; k < S::kGroups - 1; ++k)
#pragma unroll
            for (int i = 0; i < kN; ++i)
#pragma unroll
                for (int j = 0; j < kM; ++j) {
                    const f32x4_v v = s_sum[((k * S::kWaves + wave) * S::kFrags + i * kM + j) * 64 + lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] += v[e];
                }
    }

    // ---- results
    if (a.splits > 1) {
        f32x4_v *p = reinterpret_cast<f32x4_v *>(a.partial) +
                     (((int64_t)tile * a.splits + split) * S::kWaves + wave) * (S::kFrags * 64) + lane;
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int j = 0; j < kM; ++j)
                if (t0 + wm + 16 * j < a.l.tokens) p[(i * kM + j) * 64] = acc[i][j];
        return;
    }
#pragma unroll
    for (int j = 0; j < kM; ++j)
#pragma unroll
        for (int i = 0; i < kN; ++i)
            store_results<GT>(a, t0 + wm + 16 * j + n, o0 + wn + 16 * i + 4 * g, acc[i][j]);
}

// Adds up the parts of split tiles, in their order: a thread has four results.
template <int GT, class S>
__global__ __launch_bounds__(256) void k_qsdp_tile_join(TileArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // tile, wave, frag
    const int frag = (int)(item % S::kFrags), wave = (int)(item / S::kFrags % S::kWaves);
    const int64_t tile = item / (S::kFrags * S::kWaves);
    if (tile >= (int64_t)a.tiles_m * a.tiles_n) return;
    constexpr int kM = S::WM / 16;
    const int64_t t = tile % a.tiles_m * S::TM + (wave % (S::TM / S::WM)) * S::WM + 16 * (frag % kM) + (lane & 15);
    const int64_t o = tile / a.tiles_m * S::TN + (wave / (S::TM / S::WM)) * S::WN + 16 * (frag / kM) + 4 * (lane >> 4);
    if (t >= a.l.tokens || o >= a.width) return;
    const f32x4_v *p = reinterpret_cast<const f32x4_v *>(a.partial) +
                       ((tile * a.splits * S::kWaves + wave) * S::kFrags + frag) * 64 + lane;
    constexpr int64_t kStep = S::kWaves * S::kFrags * 64;
    f32x4_v v = *p;
    // four parts at a time, so that a wait is for four (behind the last one: the last one, not used)
    for (int s = 1; s < a.splits; s += 4) {
        f32x4_v q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = p[min(s + k, a.splits - 1) * kStep];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s + k < a.splits) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += q[k][e];
            }
    }
    store_results<GT>(a, t, o, v);
}

}  // namespace onebit
