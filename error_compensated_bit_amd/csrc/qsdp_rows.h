// qsdp_rows.h -- few rows times a coded matrix: bound by reading the codes, once.
//   out_{t,o} = sum_b [ delta_b sum_{i in b} x_{t,i} c_i + min_b sum_{i in b} x_{t,i} ]
// with the sums over a bucket's part of row o.  Codes enter the matrix cores as whole
// numbers (4 bits: 16 + c, by a shift and a mask for two; 8 bits: c, or c - 128 in fp16), and
// what the offset adds is taken back through the bucket's minimum: min' = fl32(min - offset *
// delta).  Beside that nothing but the fp32 sums and the result is rounded.  The sums of x
// alone come from one more product, with ones.
//
// v_mfma_f32_16x16x32 with x's rows along the first side and rows of the matrix along the
// second: a lane holds one matrix row's results, so it needs the deltas of that row only.
// A wave takes 16 * NT rows of the matrix, 128 columns a step, four steps ahead in registers: whole
// cache lines of eight rows at a time (half lines of 16 rows run at two thirds of the rate),
// which LDS turns into the operands' order.  The waves of a group share the columns and with
// them x, which goes through LDS too; groups share the columns of the same rows among them and
// add up in LDS at the end.
//
// Measured (a copy moves 4.8 to 4.95 TB/s): 32 tokens over 28672 x 8192, 4 bits, 48 to 52 us for 134 MB (2.7
// TB/s), 54 with codes that no cache holds; 5 over 50257 x 1600, 8 bits, buckets of 1024, 25 to 28 us for 82 MB
// (cold 28); one over 8192 x 8192, 4 bits, 15 us for 38 MB (cold 17), over 6400 x 1600 6.0 to 6.7 us, of which a
// launch is 4.  Without its products the first takes 40, the second 26: what the loop reads, 128 bytes of eight
// rows at a time, comes at 3.1 to 3.3 TB/s (alone, in a probe, 5).  The matrix cores are busy in 23% and 11% of the
// compute units' time, LDS in 31% and 33%.
#pragma once

#include "qsdp_linear.h"

namespace onebit {

constexpr int kRowsChunk = 128;  // columns of a step
constexpr int kRowsAhead = 4;    // steps under way

// What stands in front of a code in the operand, and so in every sum over codes.
template <int GT, int BITS>
constexpr float kCodeOffset = BITS == 4 ? 16.0f : GT == kGradBF16 ? 0.0f : -128.0f;

// The mask that leaves two 4-bit codes in the mantissas of a pair, and the pair (16, 16) that goes
// in front.  The compiler must not know the numbers: from two constants it makes two
// instructions, from a scalar and a vector register one (v_and_or_b32).
struct CodeMask {
    uint32_t mask, offset;
};
template <int GT>
__device__ __forceinline__ CodeMask code_mask() {
    CodeMask m;
    m.mask = GT == kGradBF16 ? 0x00780078u : 0x03c003c0u;
    m.offset = GT == kGradBF16 ? 0x41804180u : 0x4c004c00u;
    asm volatile("" : "+s"(m.mask));
    asm volatile("" : "+v"(m.offset));
    return m;
}

// Eight consecutive codes as an operand.  4 bits (w0): elements 0 4, 1 5, 2 6, 3 7 of the eight,
// each in the mantissa of 16 (ulp 2^-3 in bf16, 2^-6 in fp16).  8 bits (w0, w1): in order.
template <int GT, int BITS>
__device__ __forceinline__ u32x4_v code_operand(uint32_t w0, uint32_t w1, const CodeMask &cm) {
    u32x4_v r;
    if (BITS == 4 && GT == kGradBF16) {
        r.x = ((w0 << 3) & cm.mask) | cm.offset;
        r.y = ((w0 >> 1) & cm.mask) | cm.offset;
        r.z = ((w0 >> 5) & cm.mask) | cm.offset;
        r.w = ((w0 >> 9) & cm.mask) | cm.offset;
    } else if (BITS == 4) {
        r.x = ((w0 << 6) & cm.mask) | cm.offset;
        r.y = ((w0 << 2) & cm.mask) | cm.offset;
        r.z = ((w0 >> 2) & cm.mask) | cm.offset;
        r.w = ((w0 >> 6) & cm.mask) | cm.offset;
    } else if (GT == kGradBF16) {
        // 0 .. 255 are eight bits of mantissa: the upper half of the binary32 number
        const uint32_t w[2] = {w0, w1};
        uint32_t p[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float a = (float)(w[k] & 255u), b = (float)((w[k] >> 8) & 255u);
            const float c = (float)((w[k] >> 16) & 255u), d = (float)(w[k] >> 24);
            p[2 * k] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
            p[2 * k + 1] = __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x07060302u);
        }
        r = (u32x4_v){p[0], p[1], p[2], p[3]};
    } else {
        // 1024 + c, less 1152
        const f16x2_v off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
        const uint32_t w[2] = {w0, w1};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t p = __builtin_amdgcn_perm(0x64646464u, w[k >> 1], k & 1 ? 0x04030402u : 0x04010400u);
            r[k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_v, p) + off);
        }
    }
    return r;
}

// The matching operand of eight consecutive values of x.
template <int BITS>
__device__ __forceinline__ u32x4_v x_operand(const uint4 &x) {
    if (BITS == 8) return (u32x4_v){x.x, x.y, x.z, x.w};
    return (u32x4_v){__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                     __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

// Words that the four quarters of the wave hold, each 16 consecutive bytes of a row's 64, on their way to
// where a product over 32 columns wants them.  4 bits: word j of quarter g becomes word g of
// quarter j, as products 0 .. 3 take bytes 16 j .. 16 j + 15, four of a quarter.  8 bits: products 0 and
// 1 take bytes 32 j .. 32 j + 31, eight (two words) of a quarter.
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
template <int BITS>
__device__ __forceinline__ void spread(uint4 &w) {
    if (BITS == 4) {
        swap32(w.x, w.z);
        swap32(w.y, w.w);
        swap16(w.x, w.y);
        swap16(w.z, w.w);
    } else {
        // pairs of words (x, y) and (z, w): the pair 2 g + h of the row belongs to product (2 g + h) / 4
        swap16(w.x, w.z);
        swap16(w.y, w.w);
        swap32(w.x, w.z);
        swap32(w.y, w.w);
    }
}

// the value that lane `lane` holds
__device__ __forceinline__ float from_lane(int lane, float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_ds_bpermute(4 * lane, (int)__float_as_uint(v)));
}

// GROUPS: the columns of a step have up to so many buckets of a row, 128 / GROUPS columns each (4 or 1).
// WAVES of a group, SPLIT groups.
template <int GT, int BITS, int GROUPS, int NT, int MT, int WAVES, int SPLIT>
__global__ __launch_bounds__(64 * WAVES * SPLIT) void k_qsdp_rows(LinearArgs a) {
    constexpr int kTiles = NT * MT, kPer = 4 / GROUPS, kThreads = 64 * WAVES;
    // A load of minima and maxima brings those of four groups: of kPer steps, that is of one or of all
    // that are under way.
    constexpr int kSets = kRowsAhead / kPer;
    static_assert(kRowsAhead == 4, "sets of scales");
    // A load of codes brings 128 bytes, a cache line's worth, of 8 rows: two steps of 4-bit codes.
    constexpr int kSteps = 8 / BITS, kWords = BITS / 4;
    constexpr int kX = 4 * MT / WAVES;  // pieces of x of a thread and step
    constexpr int kXBytes = 16 * MT * kRowsChunk * 2, kCodeBytes = 16 * 128;
    constexpr int kStage = SPLIT * (2 * kXBytes + WAVES * NT * kCodeBytes), kSums = (SPLIT - 1) * WAVES * kTiles * 1024;
    __shared__ __attribute__((aligned(16))) char s_mem[kStage > kSums ? kStage : kSums];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % WAVES);
    const int group = SPLIT == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    const int n = lane & 15, g = lane >> 4;
    const int64_t row0 = ((int64_t)blockIdx.x * WAVES + wave) * (16 * NT);
    const int cols = (int)a.cols, steps = (cols + kRowsChunk - 1) / kRowsChunk;
    // this group's steps (whole loads of codes); every group goes through as many
    const int each = ((steps + SPLIT - 1) / SPLIT + kSteps - 1) / kSteps * kSteps;
    const int begin = group * each, end = min(begin + each, steps);

    // Rows by their offsets from the wave's first (behind the last row: the last one again, not
    // written), buckets by their numbers from that row's first.  Every offset fits 32 bits: 32 rows
    // of less than 2^24 codes, and buckets of at least 32.
    const int64_t first_row = uniform(min(row0, a.rows - 1));
    const uint32_t row_parts = (uint32_t)(a.cols >> 5), bucket_parts = (uint32_t)a.bucket >> 5;
    const uint32_t row_bytes = row_parts * (4 * BITS);
    const Bucket b0 = bucket_of(first_row * row_parts, bucket_parts);
    const uint8_t *codes = a.codes + first_row * row_bytes;
    const float *lo = a.lo + b0.index, *hi = a.hi + b0.index;
    uint32_t code_at[NT][2], bucket_at[NT], part[NT];  // part: 32-column parts in front of the row in its first bucket
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            code_at[t][k] = (uint32_t)(min(first_row + 16 * t + 8 * k + (lane >> 3), a.rows - 1) - first_row) * row_bytes;
        const uint32_t parts =
            b0.part + (uint32_t)(min(first_row + 16 * t + (lane >> 2), a.rows - 1) - first_row) * row_parts;
        bucket_at[t] = parts / bucket_parts;
        part[t] = parts - bucket_at[t] * bucket_parts;
    }
    // this thread's pieces of eight values of x: of rows (tx >> 4) + 4 WAVES m
    const int tx = threadIdx.x % kThreads;
    const uint16_t *x[kX];
#pragma unroll
    for (int m = 0; m < kX; ++m) x[m] = a.x + min((int64_t)(4 * WAVES * m + (tx >> 4)), a.tokens - 1) * a.x_stride;

    uint4 w[kRowsAhead][NT][kWords], xr[kRowsAhead][kX];
    float l[kSets][NT], h[kSets][NT];
    // (behind the last step: the first one's again, not used; behind the row's end its last piece, times zeros)
    const auto load = [&](int i, int slot) {
        const int s = i < end ? i : begin;
        if (slot % kSteps == 0) {
            const uint32_t in_row = min((uint32_t)s * (16 * BITS) + 16 * (lane & 7), row_bytes - 16);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    w[slot + (kSteps == 2 ? k : 0)][t][kSteps == 2 ? 0 : k] =
                        ld_stream(reinterpret_cast<const uint4 *>(codes + (code_at[t][k] + in_row)));
        }
        const int column = min(s * kRowsChunk + 8 * (tx & 15), cols - 8);
#pragma unroll
        for (int m = 0; m < kX; ++m) xr[slot][m] = *reinterpret_cast<const uint4 *>(x[m] + column);
    };
    // minima and maxima of the four groups of steps i .. i + kPer - 1, group q of row r in lane 4 r + q
    // (behind the row's end the row's last)
    const auto load_scales = [&](int i, int set) {
        const uint32_t c = min((uint32_t)(i * 4 + (lane & 3) * kPer), row_parts - 1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t k = part[t] + c;
            const uint32_t b = bucket_at[t] + (bucket_parts == 1 ? k : __umulhi(k, a.bucket_magic));
            l[set][t] = lo[b];
            h[set][t] = hi[b];
        }
    };
    // x of a step in LDS: rows of 256 bytes, the 16-byte pieces of row r in the order p ^ r, so that the same
    // piece of 16 rows lies in different banks; zeros behind the row's end
    u32x4_v *s_x = reinterpret_cast<u32x4_v *>(s_mem + group * 2 * kXBytes);
    const auto keep_x = [&](int i, int slot) {
        const bool in = GROUPS == 1 || i * kRowsChunk + 8 * (tx & 15) < cols;
        const u32x4_v none = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int m = 0; m < kX; ++m) {
            const int r = 4 * WAVES * m + (tx >> 4);
            s_x[(i & 1) * (kXBytes / 16) + 16 * r + ((tx & 15) ^ (r & 15))] = in ? x_operand<BITS>(xr[slot][m]) : none;
        }
    };
    // Codes as they were loaded, eight pieces of a row in neighbouring lanes, go through LDS to the lanes that
    // the matrix cores want them in: pieces g and 4 + g of row n in lane n + 16 g.  Each wave its own.
    u32x4_v *s_w = reinterpret_cast<u32x4_v *>(s_mem + SPLIT * 2 * kXBytes + (group * WAVES + wave) * NT * kCodeBytes);
    const auto turn_codes = [&](int slot) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 &v = w[slot + (kSteps == 2 ? k : 0)][t][kSteps == 2 ? 0 : k];
                s_w[128 * t + 64 * k + (lane ^ (lane >> 3))] = (u32x4_v){v.x, v.y, v.z, v.w};
            }
        // (what other lanes wrote is read: nothing else tells the compiler of the order)
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const u32x4_v v = s_w[128 * t + 8 * n + ((4 * k + g) ^ (n & 7))];
                w[slot + (kSteps == 2 ? k : 0)][t][kSteps == 2 ? 0 : k] = make_uint4(v.x, v.y, v.z, v.w);
            }
    };

    f32x4_v acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = (f32x4_v){0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t one = GT == kGradBF16 ? 0x3f803f80u : 0x3c003c00u;
    const u32x4_v ones = {one, one, one, one};
    const f32x4_v zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const CodeMask cm = code_mask<GT>();

    // set: the first of the step's groups among the four whose scales are at hand
    const auto multiply = [&](int i, int slot, const float (&delta)[NT][4], const float (&base)[NT][4], int set) {
        const u32x4_v *xs_of = s_x + (i & 1) * (kXBytes / 16) + 16 * n;
        if (GROUPS > 1) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < kWords; ++k) spread<BITS>(w[slot][t][k]);
        }
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) {
            f32x4_v sum[NT][MT], xs[MT];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                // The product's columns: with several groups the part's own 32; else those that the
                // quarters hold, eight each.
                const int j = u * kPer + k;
                const int piece = GROUPS > 1 ? 4 * j + g : BITS == 4 ? 4 * g + j : 8 * (j >> 1) + 2 * g + (j & 1);
                u32x4_v xo[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    xo[m] = xs_of[256 * m + (piece ^ n)];
                    xs[m] = product16<GT>(xo[m], ones, k == 0 ? zero : xs[m]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 &v = w[slot][t][BITS == 4 ? 0 : j >> 1];
                    const uint32_t w0 = BITS == 4 ? (j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w) : (j & 1 ? v.z : v.x);
                    const u32x4_v c = code_operand<GT, BITS>(w0, BITS == 4 ? 0u : j & 1 ? v.w : v.y, cm);
#pragma unroll
                    for (int m = 0; m < MT; ++m) sum[t][m] = product16<GT>(xo[m], c, k == 0 ? zero : sum[t][m]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[t][m][e] = fmaf(delta[t][set + u], sum[t][m][e], fmaf(base[t][set + u], xs[m][e], acc[t][m][e]));
        }
    };

#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) {
        if (k % kPer == 0) load_scales(begin + k, k / kPer);
        load(begin + k, k);
    }
    float delta[NT][4], base[NT][4];
    for (int i = begin; i < begin + each; i += kRowsAhead) {
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            if (i + u >= begin + each) break;
            keep_x(i + u, u);
            if (u % kSteps == 0) turn_codes(u);
            __syncthreads();
            if (u % kPer == 0) {
                const int k = u / kPer;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float d = bucket_delta<BITS>(l[k][t], h[k][t]);
                    const float b = fmaf(-kCodeOffset<GT, BITS>, d, l[k][t]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        delta[t][q] = from_lane(4 * n + q, d);
                        base[t][q] = from_lane(4 * n + q, b);
                    }
                }
                load_scales(i + u + kRowsAhead, k);
            }
            if (i + u < end) multiply(i + u, u, delta, base, (u % kPer) * GROUPS);
            if (u % kSteps == kSteps - 1) {
#pragma unroll
                for (int k = kSteps - 1; k >= 0; --k) load(i + u - k + kRowsAhead, u - k);
            }
        }
    }

    // ---- the groups' sums, in their order
    if (SPLIT > 1) {
        float *s_sum = reinterpret_cast<float *>(s_mem);
        __syncthreads();
        if (group > 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s_sum[((((group - 1) * WAVES + wave) * kTiles + t * MT + m) * 4 + e) * 64 + lane] = acc[t][m][e];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int s = 0; s < SPLIT - 1; ++s)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[t][m][e] += s_sum[(((s * WAVES + wave) * kTiles + t * MT + m) * 4 + e) * 64 + lane];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t o = row0 + 16 * t + n;
        if (o >= a.rows) continue;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int token = 16 * m + 4 * g + e;
                if (token < a.tokens) a.out[token * a.out_stride + o] = (uint16_t)round_pair<GT>(acc[t][m][e], 0.0f);
            }
    }
}

}  // namespace onebit
