// kvq_step.h -- attention of few query rows over the coded cache (a token or some
// drafts for each sequence): bound by reading the cache, once for 16 query rows of a cache
// head (or 32, where the caller's tables are for long caches), again for the next.
//
// A wave takes 32 tokens at a time straight from memory into the operands' registers,
// no LDS and no barrier in the loop.  S^T = K Q^T: the lane that holds a query row in
// S^T holds it again in P^T, the right operand of O^T = V^T P^T, so the weights never
// move between lanes; which tokens a lane's eight places stand for is free as long as
// V^T's operand agrees.  v_mfma_f32_16x16x32_f16 with tokens (then dimensions) along
// the first side and query rows (tokens x heads of one cache head) along the second.
//
// The work of a launch is one line of units of 128 tokens (sequence by sequence, head
// by head); every workgroup takes an equal stretch of it, so sequences of any lengths
// share the GPU evenly.  What a stretch covers of a sequence and head only in part is
// left as a partial result, and the last of its workgroups to arrive joins them, in
// the order of the line.
//
// Measured: 64 sequences of 100 to 16000 tokens, 8 heads of 128, 4 bits, 155 us for
// 0.67 GB (4.3 TB/s; a copy moves 4.8); 2 of 131072, 8 bits, 126 us (4.4 TB/s); 24 x 5
// drafts over 900 to 5000, 16 heads of 64, 36 us (4.4 TB/s).  A single sequence of
// 1000 tokens takes 11 us, waits for memory one after the other.
#pragma once

#include "kvq_attention.h"

namespace onebit {

constexpr int kStepWaves = 4;
constexpr int kStepBlock = 64 * kStepWaves;
constexpr int kStepUnit = 32 * kStepWaves;  // tokens
constexpr int kStepSeqs = 1024;             // sequences of one launch
constexpr int kStepMaxGroups = 2048;        // workgroups of one launch
constexpr int kStepHeader = 4 * kStepMaxGroups;  // bytes of counters in front of the partial results
constexpr int kJoin = 8;                    // partial results that a join reads at once

// A weight may exceed the running maximum's by 2^8 before the sums are rescaled.
constexpr float kSlack = 8.0f;

template <int D, int NT>
struct StepPartial {
    float o[16 * NT][D];
    float ml[16 * NT][2];  // maximum and sum of weights
};

// Partial results pass between workgroups through agent-scope accesses only, which go
// past the caches of one XCD: a release fence would write the whole L2 of an XCD back,
// for every workgroup that leaves one (measured: 284 us instead of 120 for 24
// sequences of 16 heads).
__device__ __forceinline__ void st_agent2(float *p, float a, float b) {
    st_agent(reinterpret_cast<uint64_t *>(p), (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32));
}
__device__ __forceinline__ float2 ld_agent2(const float *p) {
    const uint64_t v = ld_agent(reinterpret_cast<const uint64_t *>(p));
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
// all of this wave's stores have reached where the other XCDs see them
__device__ __forceinline__ void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ float over_quarters_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float over_quarters_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

template <int D, int BITS>
struct StepTile {
    static constexpr int kRow = D * BITS / 8;                  // bytes of a row
    static constexpr int kPieces = kRow >= 64 ? kRow / 64 : 1;  // loads of a key row by its four lanes
    static constexpr int kPieceWords = kRow >= 64 ? 4 : 2;
    static constexpr int kSteps = D / 32;                      // products over dimensions
    static constexpr int kStepWords = BITS / 4;                // words of a step
    static constexpr int kDims = D / 16;                       // value dimensions of a lane
    static constexpr int kValBytes = kRow / 16;
    static constexpr int kValWords = kValBytes >= 4 ? kValBytes / 4 : 1;
    // first dimension of step `s` in quarter `c` of the wave
    static __device__ __forceinline__ int dim_of(int s, int c) {
        constexpr int per_lane = kPieceWords * 32 / BITS, per_piece = kPieceWords / kStepWords;
        return (s / per_piece) * 4 * per_lane + c * per_lane + (s % per_piece) * 8;
    }
    // a quarter's share of 16 key rows: lane % 16 is the row
    static __device__ __forceinline__ void load_keys(const uint8_t *rows, int lane, uint32_t (&w)[kPieces * kPieceWords]) {
        const uint8_t *p = rows + (lane & 15) * kRow + (lane >> 4) * (4 * kPieceWords);
        if (kPieceWords == 4) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p + 64 * i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x; w[1] = v.y;
        }
    }
    // kDims consecutive dimensions of four value rows: lane % 16 counts the dimensions'
    // groups, lane / 16 the rows' groups of four
    static __device__ __forceinline__ void load_values(const uint8_t *rows, int lane, uint32_t (&w)[4][kValWords]) {
        const uint8_t *p = rows + (lane >> 4) * (4 * kRow) + (lane & 15) * kValBytes;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *s = p + j * kRow;
            if (kValBytes == 16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(s);
                w[j][0] = v.x; w[j][1 % kValWords] = v.y; w[j][2 % kValWords] = v.z; w[j][3 % kValWords] = v.w;
            } else if (kValBytes == 8) {
                const uint2 v = *reinterpret_cast<const uint2 *>(s);
                w[j][0] = v.x; w[j][1 % kValWords] = v.y;
            } else if (kValBytes == 4) {
                w[j][0] = *reinterpret_cast<const uint32_t *>(s);
            } else {
                w[j][0] = *reinterpret_cast<const uint16_t *>(s);
            }
        }
    }
};

template <int GT, int D, int BITS, int NT>
__global__ __launch_bounds__(kStepBlock, NT == 1 && D <= 128 ? 3 : 2) void k_kvq_step(KvqAttnArgs a) {
    using T = StepTile<D, BITS>;
    constexpr int kRows = 16 * NT;
    // the codes' offset as the operands hold it
    constexpr float kOffset = (float)KvqLevels<BITS>::kZero / (float)(1 << kCodeShift<BITS>);
    __shared__ int64_t s_pre[kStepSeqs + 1];
    __shared__ float s_o[kStepWaves][16][D + 4];
    __shared__ float s_m[kStepWaves][kRows], s_l[kStepWaves][kRows];
    __shared__ int64_t s_scan[kStepWaves];
    __shared__ int s_last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, c = lane >> 4;

    // ---- units of every sequence, as running sums
    {
        constexpr int kPer = kStepSeqs / kStepBlock;
        int64_t u[kPer], sum = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int b = threadIdx.x * kPer + k;
            u[k] = 0;
            if (b < a.batch) {
                const KvqSeq s = kvq_seq(a, b);
                const int64_t rows = (int64_t)s.len * a.group;
                if (rows > 0 && rows <= a.max_rows) {
                    const int lo = kvq_lo(a, s, 0) & ~31;
                    u[k] = ((rows + kRows - 1) / kRows) * a.c.heads *
                           max(1, (max(s.kv - lo, 0) + kStepUnit - 1) / kStepUnit);
                }
            }
            sum += u[k];
        }
        int64_t incl = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t t = __shfl_up(incl, d, 64);
            if (lane >= d) incl += t;
        }
        if (lane == 63) s_scan[wave] = incl;
        __syncthreads();
        for (int w = 0; w < wave; ++w) incl += s_scan[w];
        int64_t at = incl - sum;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            s_pre[threadIdx.x * kPer + k] = at;
            at += u[k];
        }
        if (threadIdx.x == kStepBlock - 1) s_pre[kStepSeqs] = at;
        __syncthreads();
    }
    const int64_t total = uniform(s_pre[kStepSeqs]);
    const int64_t groups = min((int64_t)gridDim.x, total);
    if ((int64_t)blockIdx.x >= groups) return;
    // the first `more` workgroups take one unit more than the others
    const int64_t each = udiv(total, groups), more = total - each * groups;
    const auto begin_of = [&](int64_t w) { return w * each + min(w, more); };
    const int64_t end = begin_of((int64_t)blockIdx.x + 1);
    int64_t pos = begin_of(blockIdx.x);
    int b;
    {
        int lo = 0, hi = kStepSeqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] <= pos) lo = mid; else hi = mid;
        }
        b = uniform(lo);
    }
    uint32_t *counters = static_cast<uint32_t *>(a.workspace);
    StepPartial<D, NT> *parts =
        reinterpret_cast<StepPartial<D, NT> *>(static_cast<char *>(a.workspace) + kStepHeader);

    for (bool first = true; pos < end; first = false) {
        while (s_pre[b + 1] <= pos) ++b;
        b = uniform(b);
        KvqSeq seq = kvq_seq(a, b);
        seq.q0 = uniform(seq.q0);
        seq.len = uniform(seq.len);
        seq.kv = uniform(seq.kv);
        const int64_t seq_begin = uniform(s_pre[b]);
        const int rows = seq.len * a.group;
        const int base = kvq_lo(a, seq, 0) & ~31;
        const int per_item = max(1, (max(seq.kv - base, 0) + kStepUnit - 1) / kStepUnit);
        const int item = uniform((int)udiv(pos - seq_begin, per_item));
        const int64_t item_begin = seq_begin + (int64_t)item * per_item, item_end = item_begin + per_item;
        const int64_t seg_end = min(end, item_end);
        const int rt = item / a.c.heads, g = item % a.c.heads;
        const int r0 = rt * kRows, r1 = min(rows, r0 + kRows);
        const int t0 = r0 / a.group, t1 = (r1 - 1) / a.group;
        // the stretch's tokens that some row of the tile attends to
        const int from = max(base + (int)(pos - item_begin) * kStepUnit, kvq_lo(a, seq, t0) & ~31);
        const int to = (int)min((int64_t)kvq_hi(seq, t1), base + (seg_end - item_begin) * kStepUnit);
        // tokens that all rows attend to
        const int all_lo = kvq_lo(a, seq, t1), all_hi = kvq_hi(seq, t0);

        // ---- queries
        f16x8_v qf[NT][T::kSteps];
        float qs[NT], q_off[NT];
        int hi[NT], lo[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = r0 + 16 * nt + n;
            const bool live = r < r1;
            const int t = live ? r / a.group : t0, h = live ? g * a.group + r % a.group : 0;
            lo[nt] = kvq_lo(a, seq, t);
            hi[nt] = kvq_hi(seq, t);
            const uint16_t *src = a.q + (int64_t)(seq.q0 + t) * a.q_token_stride + (int64_t)h * a.q_head_stride;
            uint4 raw[T::kSteps];
#pragma unroll
            for (int s = 0; s < T::kSteps; ++s)
                raw[s] = live ? *reinterpret_cast<const uint4 *>(src + T::dim_of(s, c)) : make_uint4(0, 0, 0, 0);
            float amax = 0.0f;
#pragma unroll
            for (int s = 0; s < T::kSteps; ++s) {
                const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    amax = fmaxf(amax, fmaxf(fabsf(half_bits_to_float<GT>(w[k] & 0xffffu)),
                                             fabsf(half_bits_to_float<GT>(w[k] >> 16))));
            }
            const int kq = query_exponent(over_quarters_max(amax));
            const float up = __uint_as_float(__float_as_uint(pow2(kq)) ^ a.q_sign);
            float sum = 0.0f;
#pragma unroll
            for (int s = 0; s < T::kSteps; ++s) {
                const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
                float f[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = half_bits_to_float<GT>(w[k] & 0xffffu);
                    f[2 * k + 1] = half_bits_to_float<GT>(w[k] >> 16);
                }
                qf[nt][s] = query_operand<BITS>(f, up);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += f[k] * up;
            }
            q_off[nt] = -kOffset * over_quarters_sum(sum);
            qs[nt] = ldexpf(a.scale2, kCodeShift<BITS> - kq);
            if (a.cap2 > 0.0f) qs[nt] *= a.cap_scale;
        }

        // ---- the loop over this wave's tiles of 32 tokens
        f32x4_v o[NT][T::kDims];
        float m[NT], l[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = kNone;
            l[nt] = 0.0f;
#pragma unroll
            for (int u = 0; u < T::kDims; ++u) o[nt][u] = (f32x4_v){0.0f, 0.0f, 0.0f, 0.0f};
        }
        // A row's value scales are taken times 2^kv_exp, chosen for the largest that the row itself
        // attends to: what other rows of the tile attend to must not decide what fp16 loses of its weights.
        int kv_exp[NT];
        float v_top[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            kv_exp[nt] = 126;
            v_top[nt] = 0.0f;
        }
        const int32_t *table = a.table + (int64_t)b * a.table_stride;
        // page number of token j, and the cache row of token j (a multiple of 16); without branches,
        // where the compiler would wait for all loads under way.  Tokens behind the table's end
        // get its last page (they are masked); a page outside the cache gives rows of page 0, to be
        // left out.
        const int last_page = (a.max_tokens >> a.c.shift) - 1;
        const uint32_t in_cache = (uint32_t)min(a.c.n_pages, (int64_t)1 << 31);
        const auto page_of = [&](int j) -> int { return table[min(j >> a.c.shift, last_page)]; };
        const auto row_of = [&](int page, int j, bool &ok) -> int64_t {
            page = uniform(page);
            ok = (uint32_t)page < in_cache;
            return (int64_t)((((uint64_t)(uint32_t)(ok ? page : 0) * (uint32_t)a.c.heads + (uint32_t)g) << a.c.shift) |
                             (uint32_t)(j & (a.c.page - 1)));
        };
        uint32_t kw[2][T::kPieces * T::kPieceWords], vw[2][4][T::kValWords];
        float4 ks[2];
        int64_t row[2];
        bool ok[2];
        int pages[2];
        int j = from + 32 * wave;
        if (j < to) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                row[tt] = row_of(page_of(j + 16 * tt), j + 16 * tt, ok[tt]);
                T::load_keys(a.c.codes[0] + row[tt] * T::kRow, lane, kw[tt]);
                ks[tt] = *reinterpret_cast<const float4 *>(a.c.scales[0] + row[tt] + 4 * c);
            }
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) pages[tt] = page_of(j + kStepUnit + 16 * tt);
        }
        for (; j < to; j += kStepUnit) {
            float4 vs[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                vs[tt] = *reinterpret_cast<const float4 *>(a.c.scales[1] + row[tt] + 4 * c);
                T::load_values(a.c.codes[1] + row[tt] * T::kRow, lane, vw[tt]);
            }
            f32x4_v acc[NT][2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[nt][tt] = (f32x4_v){q_off[nt], q_off[nt], q_off[nt], q_off[nt]};
#pragma unroll
                for (int s = 0; s < T::kSteps; ++s) {
                    const f16x8_v kf =
                        codes_over_dims<BITS>(kw[tt][s * T::kStepWords], kw[tt][s * T::kStepWords + (BITS == 8 ? 1 : 0)]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        acc[nt][tt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[nt][s], acc[nt][tt], 0, 0, 0);
                }
            }
            const bool whole = j >= all_lo && j + 32 <= all_hi && ok[0] && ok[1];
            const bool page_ok[2] = {ok[0], ok[1]};
            const auto attends = [&](int nt, int k) {  // to the lane's token k
                const int t = j + 16 * (k >> 2) + 4 * c + (k & 3);
                return page_ok[k >> 2] && t >= lo[nt] && t < hi[nt];
            };
            // (an infinite scale becomes NaN here: the score of its token may not come out -inf, of weight 0,
            // nor go under a cap)
            float kscale[2][4] = {{ks[0].x, ks[0].y, ks[0].z, ks[0].w}, {ks[1].x, ks[1].y, ks[1].z, ks[1].w}};
#pragma unroll
            for (int k = 0; k < 8; ++k) kscale[k >> 2][k & 3] = fmaf(kscale[k >> 2][k & 3], 0.0f, kscale[k >> 2][k & 3]);
            // the next tile's keys are on their way from here on (behind the last tile: of rows
            // that exist and are not used)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) row[tt] = row_of(pages[tt], j + kStepUnit + 16 * tt, ok[tt]);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) pages[tt] = page_of(j + 2 * kStepUnit + 16 * tt);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                T::load_keys(a.c.codes[0] + row[tt] * T::kRow, lane, kw[tt]);
                ks[tt] = *reinterpret_cast<const float4 *>(a.c.scales[0] + row[tt] + 4 * c);
            }
            // scores in units of log2(e)
            float x[NT][8];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float top = kNone;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float y = acc[nt][k >> 2][k & 3] * kscale[k >> 2][k & 3] * qs[nt];
                    if (a.cap2 > 0.0f) y = a.cap2 > kWideCap2 ? capped_wide(y, a.cap2) : capped(y, a.cap2);
                    if (!whole && !attends(nt, k)) y = kNone;
                    x[nt][k] = y;
                    top = fmaxf(top, y);
                }
                grow |= top > m[nt] + kSlack;
            }
            if (__any(grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float top = x[nt][0];
#pragma unroll
                    for (int k = 1; k < 8; ++k) top = fmaxf(top, x[nt][k]);
                    top = over_quarters_max(top);
                    // (each row by its own scores: its roundings do not depend on the other rows')
                    const float f = top > m[nt] + kSlack ? exp2_fast(m[nt] - top) : 1.0f;
                    m[nt] = top > m[nt] + kSlack ? top : m[nt];
                    l[nt] *= f;
#pragma unroll
                    for (int u = 0; u < T::kDims; ++u) o[nt][u] *= f;
                }
            }
            const float vscale[2][4] = {{vs[0].x, vs[0].y, vs[0].z, vs[0].w}, {vs[1].x, vs[1].y, vs[1].z, vs[1].w}};
            float v_size[8], v_new[NT];  // an infinite scale of one token must not set the others' range
            bool rise = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float v = fabsf(vscale[k >> 2][k & 3]);
                v_size[k] = v < INFINITY ? v : 0.0f;
            }
            if (whole) {
                float v = v_size[0];
#pragma unroll
                for (int k = 1; k < 8; ++k) v = fmaxf(v, v_size[k]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) v_new[nt] = v;
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    v_new[nt] = 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v_new[nt] = fmaxf(v_new[nt], attends(nt, k) ? v_size[k] : 0.0f);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) rise |= v_new[nt] > v_top[nt];
            if (__any(rise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    v_top[nt] = fmaxf(v_top[nt], over_quarters_max(v_new[nt]));
                    const int e = value_exponent(v_top[nt]);
#pragma unroll
                    for (int u = 0; u < T::kDims; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[nt][u][i] = ldexpf(o[nt][u][i], e - kv_exp[nt]);
                    kv_exp[nt] = e;
                }
            }
            f16x8_v pf[NT], pl[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t pw[4], lw[4];
                const float vf = pow2(kv_exp[nt]);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    float e[2], p[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        e[i] = exp2_fast(x[nt][k + i] - m[nt]);
                        p[i] = e[i] * (vscale[k >> 2][(k & 3) + i] * vf);
                        if (!whole) {  // (tokens that the row does not attend to may hold anything)
                            const bool in = attends(nt, k + i);
                            e[i] = in ? e[i] : 0.0f;
                            p[i] = in ? p[i] : 0.0f;
                        }
                        l[nt] += e[i];
                    }
                    pw[k >> 1] = round_pair<kGradF16>(p[0], p[1]);
                    if (kTwoPart<GT>) lw[k >> 1] = rest_pair(p[0], p[1], pw[k >> 1]);
                }
                pf[nt] = __builtin_bit_cast(f16x8_v, (u32x4_v){pw[0], pw[1], pw[2], pw[3]});
                if (kTwoPart<GT>) pl[nt] = __builtin_bit_cast(f16x8_v, (u32x4_v){lw[0], lw[1], lw[2], lw[3]});
            }
#pragma unroll
            for (int u = 0; u < T::kDims; ++u) {
                const int w = u * BITS / 32;
                const f16x2_v unit = splat16(kUnitScale<BITS>), zero = splat16(-kUnitOffset<BITS>);
                const u32x4_v av = {fma16(code_pair<BITS>(vw[0][0][w], vw[0][1][w], u), unit, zero),
                                    fma16(code_pair<BITS>(vw[0][2][w], vw[0][3][w], u), unit, zero),
                                    fma16(code_pair<BITS>(vw[1][0][w], vw[1][1][w], u), unit, zero),
                                    fma16(code_pair<BITS>(vw[1][2][w], vw[1][3][w], u), unit, zero)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    o[nt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_v, av), pf[nt], o[nt][u], 0, 0, 0);
                    if (kTwoPart<GT>)
                        o[nt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_v, av), pl[nt], o[nt][u], 0, 0, 0);
                }
            }
        }

        // ---- the waves' results, joined in LDS
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] = over_quarters_sum(l[nt]);
            if (c == 0) {
                s_m[wave][16 * nt + n] = m[nt];
                s_l[wave][16 * nt + n] = l[nt];
            }
        }
        __syncthreads();
        const bool alone = pos == item_begin && seg_end == item_end;
        const int slot = 2 * blockIdx.x + (first ? 0 : 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 16 * nt + n;
            float mm = s_m[0][r], ll = 0.0f;
#pragma unroll
            for (int w = 1; w < kStepWaves; ++w) mm = fmaxf(mm, s_m[w][r]);
#pragma unroll
            for (int w = 0; w < kStepWaves; ++w) ll += s_l[w][r] * exp2_fast(s_m[w][r] - mm);
            // normalised here, so that nothing overflows whatever the values' size
            const float f = ll != 0.0f ? exp2_fast(m[nt] - mm) / ll : 0.0f;
            float *dst = &s_o[wave][n][4 * c];
#pragma unroll
            for (int u = 0; u < T::kDims; ++u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[nt][u][i] = ldexpf(o[nt][u][i] * f, kUnitShift - kv_exp[nt]);
                }
                *reinterpret_cast<f32x4_v *>(dst + 16 * u) = o[nt][u];
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 16 * D / 4; i += kStepBlock) {
                const int rr = i / (D / 4), d = 4 * (i % (D / 4));
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = ((d + k) % T::kDims) * 16 + (d + k) / T::kDims;
                    v[k] = (s_o[0][rr][at] + s_o[1][rr][at]) + (s_o[2][rr][at] + s_o[3][rr][at]);
                }
                const int r_out = r0 + 16 * nt + rr;
                if (r_out >= r1) continue;
                if (alone) {
                    const int64_t to_row = (int64_t)(seq.q0 + r_out / a.group) * a.q_heads + g * a.group + r_out % a.group;
                    store_out4<GT>(a.out + to_row * D + d, v);
                } else {
                    st_agent2(&parts[slot].o[16 * nt + rr][d], v[0], v[1]);
                    st_agent2(&parts[slot].o[16 * nt + rr][d + 2], v[2], v[3]);
                }
            }
            if (wave == 0 && c == 0 && r0 + r < r1) {
                if (alone) {
                    if (a.lse) {
                        const int rr = r0 + r;
                        a.lse[(int64_t)(seq.q0 + rr / a.group) * a.q_heads + g * a.group + rr % a.group] =
                            ll != 0.0f ? (mm + log2f(ll)) * 0.693147180559945f : -INFINITY;
                    }
                } else {
                    st_agent2(parts[slot].ml[r], mm, ll);
                }
            }
            __syncthreads();
        }

        // ---- the last of an item's workgroups joins the partial results
        if (!alone) {
            const auto owner = [&](int64_t unit) {
                const int64_t at = more * (each + 1);
                return uniform((int)(unit < at ? udiv(unit, each + 1) : more + udiv(unit - at, each)));
            };
            const int w0 = owner(item_begin), w1 = owner(item_end - 1);
            wait_stores();
            __syncthreads();
            if (threadIdx.x == 0) {
                const uint32_t seen = __hip_atomic_fetch_add(&counters[w0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s_last = seen == (uint32_t)(w1 - w0);
                if (s_last) __hip_atomic_store(&counters[w0], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            __syncthreads();
            if (s_last) {
                // the item's first part is its workgroup's second stretch unless it begins there
                const int first_slot = 2 * w0 + (begin_of(w0) == item_begin ? 0 : 1);
                for (int i = threadIdx.x; i < (r1 - r0) * (D / 4); i += kStepBlock) {
                    const int r = i / (D / 4), d = 4 * (i % (D / 4));
                    float mm = kNone, ll = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    // kJoin parts on their way at a time
                    for (int w = w0; w <= w1; w += kJoin) {
                        float2 ml[kJoin], x[kJoin], y[kJoin];
#pragma unroll
                        for (int k = 0; k < kJoin; ++k) {
                            const int at = min(w + k, w1);
                            const StepPartial<D, NT> &p = parts[at == w0 ? first_slot : 2 * at];
                            ml[k] = ld_agent2(p.ml[r]);
                            x[k] = ld_agent2(&p.o[r][d]);
                            y[k] = ld_agent2(&p.o[r][d + 2]);
                        }
                        float top = mm;
#pragma unroll
                        for (int k = 0; k < kJoin; ++k) top = fmaxf(top, ml[k].x);
                        const float f0 = exp2_fast(mm - top);
                        mm = top;
                        ll *= f0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] *= f0;
#pragma unroll
                        for (int k = 0; k < kJoin; ++k) {
                            const float f = w + k <= w1 ? ml[k].y * exp2_fast(ml[k].x - mm) : 0.0f;
                            ll += f;
                            v[0] = fmaf(f, x[k].x, v[0]);
                            v[1] = fmaf(f, x[k].y, v[1]);
                            v[2] = fmaf(f, y[k].x, v[2]);
                            v[3] = fmaf(f, y[k].y, v[3]);
                        }
                    }
                    const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] *= inv;
                    const int rr = r0 + r;
                    const int64_t to_row = (int64_t)(seq.q0 + rr / a.group) * a.q_heads + g * a.group + rr % a.group;
                    store_out4<GT>(a.out + to_row * D + d, v);
                    if (a.lse && d == 0)
                        a.lse[to_row] = ll != 0.0f ? (mm + log2f(ll)) * 0.693147180559945f : -INFINITY;
                }
            }
            __syncthreads();
        }
        pos = seg_end;
    }
}

}  // namespace onebit
