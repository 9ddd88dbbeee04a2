// qsdp_tile.h -- many rows times a coded matrix or its transpose: bound by the matrix cores.
//   linear:    out_{t,o} = sum_d x_{t,d} w_{o,d}       (o a row of the matrix, d a column)
//   gradient:  out_{t,o} = sum_d x_{t,d} w_{d,o}       (o a column, d a row)
// A workgroup has TM x TN results and goes through the depth in steps of 64.  A step's x
// and its weights, expanded once for all TM rows and rounded to x's type, lie in LDS twice over:
// while one is multiplied the next is written and the one after that is on its way from memory.
// The upper half of the waves writes first and multiplies then, the lower half the other way
// round, so that of two waves on a SIMD one keeps the matrix cores busy while the other expands.
//
// LDS: rows of 64 values (128 bytes) of x and of weights, the 16-byte pieces of row r in the order
// p ^ swizzle(r); an operand of v_mfma_f32_16x16x32 is one piece of 16 rows.  Weights are the first
// operand, so that a lane holds four neighbouring results of one row of x.
#pragma once

#include "qsdp_linear.h"

namespace onebit {

constexpr int kTileDepth = 64;

template <int TM_, int TN_, int WM_, int WN_>
struct TileShape {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;
    static constexpr int kWaves = (TM / WM) * (TN / WN), kThreads = 64 * kWaves;
    static constexpr int kXPieces = TM * 8 / kThreads;  // of a thread
    static constexpr int kFrags = (WM / 16) * (WN / 16);
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

__device__ __forceinline__ int tile_swizzle(int r) { return (r ^ (r >> 3)) & 7; }

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
__global__ __launch_bounds__(S::kThreads) void k_qsdp_tile(TileArgs a) {
    constexpr int kXBytes = S::TM * 128, kWBytes = S::TN * 128;
    constexpr int kScaleBytes = GRAD ? S::kThreads * 8 : 0;
    __shared__ __attribute__((aligned(16))) char s_mem[2 * (kXBytes + kWBytes + kScaleBytes)];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    const int begin = (int)((int64_t)a.steps * split / a.splits), end = (int)((int64_t)a.steps * (split + 1) / a.splits);
    const int whole = (int)(a.depth / kTileDepth);  // steps that are full

    // ---- x: rows (tid >> 3) + kThreads / 8 * m, piece tid & 7
    const uint16_t *x[S::kXPieces];
#pragma unroll
    for (int m = 0; m < S::kXPieces; ++m)
        x[m] = a.l.x + min(t0 + (tid >> 3) + S::kThreads / 8 * m, a.l.tokens - 1) * a.l.x_stride + 8 * (tid & 7);
    u32x4_v xr[S::kXPieces];

    // ---- codes
    const int64_t row_parts = a.l.cols >> 5;
    const int64_t row_bytes = row_parts * (4 * BITS);
    const uint32_t bucket_parts = (uint32_t)a.l.bucket >> 5;
    constexpr int kCodeWords = GRAD ? 8 : BITS;  // loads of 4 rows' columns, or words of 32 codes
    uint32_t code[kCodeWords];
    float lo, hi;
    const uint8_t *codes;
    // linear: the row's first bucket and the row's place in it; gradient: those of the entry's next part
    int64_t bucket;
    uint32_t part;
    // linear: thread's row and half of a step.  gradient: rows 8 (tid / (TN / 4)) + 0 .. 7 of a step, columns
    // 4 (tid % (TN / 4)) + 0 .. 3, and an entry of the step's table of minima and steps: row tid / (TN / 32),
    // columns 32 (tid % (TN / 32)) + 0 .. 31.
    const int c_row = GRAD ? 8 * (tid / (S::TN / 4)) : tid >> 1, c_col = GRAD ? 4 * (tid % (S::TN / 4)) : 32 * (tid & 1);
    const int e_row = tid / (S::TN / 32), e_part = tid % (S::TN / 32);
    uint32_t step_parts = 0;
    int64_t step_buckets = 0;
    if (GRAD) {
        codes = a.l.codes + (min(o0 + c_col, a.l.cols - 4) * BITS >> 3);
        const int64_t p = min((o0 >> 5) + e_part, row_parts - 1);
        const Bucket b = bucket_of(((int64_t)begin * kTileDepth + e_row) * row_parts + p, bucket_parts);
        bucket = b.index;
        part = b.part;
        const Bucket d = bucket_of(kTileDepth * row_parts, bucket_parts);
        step_buckets = d.index;
        step_parts = d.part;
    } else {
        const int64_t row = min(o0 + c_row, a.l.rows - 1);
        codes = a.l.codes + row * row_bytes;
        const Bucket b = bucket_of(row * row_parts, bucket_parts);
        bucket = b.index;
        part = b.part;
    }

    // minima and maxima of step s (gradient: to be called for every step in turn)
    const auto load_scales = [&](int s) {
        if (GRAD) {
            const bool in = s < end && (int64_t)s * kTileDepth + e_row < a.l.rows;
            lo = hi = 0.0f;
            if (in) {
                lo = a.l.lo[bucket];
                hi = a.l.hi[bucket];
            }
            bucket += step_buckets;
            part += step_parts;
            if (part >= bucket_parts) {
                part -= bucket_parts;
                ++bucket;
            }
        } else {
            const int c = s * 2 + (tid & 1);
            const uint32_t k = part + (uint32_t)min((int64_t)c, row_parts - 1);
            const int64_t b = bucket + (bucket_parts == 1 ? k : __umulhi(k, a.l.bucket_magic));
            lo = a.l.lo[b];
            hi = a.l.hi[b];
            if (c >= row_parts) lo = hi = 0.0f;  // behind the row's end: weights of 0
        }
    };
    const auto load = [&](int s) {
        const int64_t d0 = (int64_t)s * kTileDepth;
        if (s < whole) {
#pragma unroll
            for (int m = 0; m < S::kXPieces; ++m) xr[m] = *reinterpret_cast<const u32x4_v *>(x[m] + d0);
        } else {
            // the depth's end: value by value, zeros behind it
#pragma unroll
            for (int m = 0; m < S::kXPieces; ++m) {
                uint32_t v[4] = {0u, 0u, 0u, 0u};
                for (int k = 0; k < 8; ++k)
                    if (d0 + 8 * (tid & 7) + k < a.depth) v[k >> 1] |= (uint32_t)x[m][d0 + k] << (16 * (k & 1));
                xr[m] = (u32x4_v){v[0], v[1], v[2], v[3]};
            }
        }
        if (GRAD) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                // (behind the last row: the last one, times a table's zeros)
                const uint8_t *p = codes + min(d0 + c_row + r, a.l.rows - 1) * row_bytes;
                code[r] = BITS == 4 ? *reinterpret_cast<const uint16_t *>(p) : *reinterpret_cast<const uint32_t *>(p);
            }
        } else {
            const int64_t d = min(d0 + c_col, a.l.cols - 32);
#pragma unroll
            for (int k = 0; k < BITS / 4; ++k) {
                const uint4 v = *reinterpret_cast<const uint4 *>(codes + (d * BITS >> 3) + 16 * k);
                code[4 * k] = v.x;
                code[4 * k + 1] = v.y;
                code[4 * k + 2] = v.z;
                code[4 * k + 3] = v.w;
            }
        }
    };

    const auto x_at = [&](int buffer) { return reinterpret_cast<u32x4_v *>(s_mem + buffer * kXBytes); };
    const auto w_at = [&](int buffer) { return reinterpret_cast<u32x4_v *>(s_mem + 2 * kXBytes + buffer * kWBytes); };
    const auto table_at = [&](int buffer) {
        return reinterpret_cast<float2 *>(s_mem + 2 * (kXBytes + kWBytes) + buffer * kScaleBytes);
    };
    const auto keep_table = [&](int buffer) { table_at(buffer)[tid] = make_float2(lo, bucket_delta<BITS>(lo, hi)); };
    const auto byte_of = [](uint32_t w, int k) -> float { return (float)((w >> (8 * k)) & 255u); };

    // x and weights of the step that has been loaded into buffer s & 1
    const auto store = [&](int s) {
        u32x4_v *xs = x_at(s & 1), *ws = w_at(s & 1);
#pragma unroll
        for (int m = 0; m < S::kXPieces; ++m) {
            const int r = (tid >> 3) + S::kThreads / 8 * m;
            xs[8 * r + ((tid & 7) ^ tile_swizzle(r))] = xr[m];
        }
        if (GRAD) {
            float w[8][4];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float2 e = table_at(s & 1)[(c_row + r) * (S::TN / 32) + (c_col >> 5)];
                float c[4];
                if (BITS == 4) {
                    // nibbles 0 2 and 1 3 as bytes
                    const uint32_t even = code[r] & 0x0f0fu, odd = (code[r] >> 4) & 0x0f0fu;
                    c[0] = byte_of(even, 0); c[1] = byte_of(odd, 0); c[2] = byte_of(even, 1); c[3] = byte_of(odd, 1);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) c[k] = byte_of(code[r], k);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) w[r][k] = __fmaf_rn(c[k], e.y, e.x);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int o = c_col + k;
                ws[8 * o + ((c_row >> 3) ^ tile_swizzle(o))] =
                    (u32x4_v){round_pair<GT>(w[0][k], w[1][k]), round_pair<GT>(w[2][k], w[3][k]),
                              round_pair<GT>(w[4][k], w[5][k]), round_pair<GT>(w[6][k], w[7][k])};
            }
        } else {
            const float delta = bucket_delta<BITS>(lo, hi);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                u32x4_v v;
                if (BITS == 4) {
                    const uint32_t even = code[p] & 0x0f0f0f0fu, odd = (code[p] >> 4) & 0x0f0f0f0fu;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = weight_pair<GT>(byte_of(even, k), byte_of(odd, k), delta, lo);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t c = code[(2 * p + (k >> 1)) % kCodeWords];
                        v[k] = weight_pair<GT>(byte_of(c, 2 * (k & 1)), byte_of(c, 2 * (k & 1) + 1), delta, lo);
                    }
                }
                ws[8 * c_row + ((4 * (tid & 1) + p) ^ tile_swizzle(c_row))] = v;
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
    const auto multiply = [&](int s) {
        const u32x4_v *xs = x_at(s & 1), *ws = w_at(s & 1);
#pragma unroll
        for (int k = 0; k < kTileDepth / 32; ++k) {
            u32x4_v wf[kN], xf[kM];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int r = wn + 16 * i + n;
                wf[i] = ws[8 * r + ((4 * k + g) ^ tile_swizzle(r))];
            }
#pragma unroll
            for (int j = 0; j < kM; ++j) {
                const int r = wm + 16 * j + n;
                xf[j] = xs[8 * r + ((4 * k + g) ^ tile_swizzle(r))];
            }
#pragma unroll
            for (int j = 0; j < kM; ++j)
#pragma unroll
                for (int i = 0; i < kN; ++i) acc[i][j] = product16<GT>(wf[i], xf[j], acc[i][j]);
        }
    };

    // ---- the pipeline
    load_scales(begin);
    if (GRAD) {
        keep_table(begin & 1);
        load_scales(begin + 1);
        __syncthreads();
    }
    load(begin);
    store(begin);
    if (GRAD) {
        keep_table((begin + 1) & 1);
        load_scales(begin + 2);
    } else if (begin + 1 < end) {
        load_scales(begin + 1);
    }
    if (begin + 1 < end) load(begin + 1);
    __syncthreads();
    const auto advance = [&](int s) {
        if (s + 1 < end) {
            store(s + 1);
            if (GRAD) {
                keep_table(s & 1);
                load_scales(s + 3);
            }
            if (s + 2 < end) {
                if (!GRAD) load_scales(s + 2);
                load(s + 2);
            }
        }
    };
    if (wave < S::kWaves / 2) {
        for (int s = begin; s < end; ++s) {
            multiply(s);
            advance(s);
            __syncthreads();
        }
    } else {
        for (int s = begin; s < end; ++s) {
            advance(s);
            multiply(s);
            __syncthreads();
        }
    }

    // ---- results
    if (a.splits > 1) {
        f32x4_v *p = reinterpret_cast<f32x4_v *>(a.partial) +
                     (((int64_t)tile * a.splits + split) * S::kWaves + wave) * (S::kFrags * 64) + lane;
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int j = 0; j < kM; ++j) p[(i * kM + j) * 64] = acc[i][j];
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
    f32x4_v v = *p;
    for (int s = 1; s < a.splits; ++s) {
        p += S::kWaves * S::kFrags * 64;
        const f32x4_v q = *p;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += q[e];
    }
    store_results<GT>(a, t, o, v);
}

}  // namespace onebit
