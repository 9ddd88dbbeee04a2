// kvq_chunk.h -- attention of chunks of new tokens over the coded cache: bound by the
// matrix products and the softmax between them.
//
// A workgroup takes 32 query rows (tokens x heads of one cache head) for each of its
// waves and walks the cache in tiles.  A tile's codes are loaded two tiles ahead,
// expanded to fp16 once for all rows while the tile before is worked on, and kept in
// LDS twice over (one barrier a tile): keys by token, values by dimension, so that
// both are read back as whole operands of v_mfma_f32_32x32x16_f16.  S^T = K Q^T and
// O^T = V^T P^T: as in the step kernel, a query row stays in its lane from the scores
// to the output.
//
// Keys are expanded to the codes (c - z) themselves, exact, and their scales are applied to
// the scores in fp32: a scale rounded to fp16 moves all of a token's score by up to one part in
// 2^11, a quarter of a weight where scores are around 500, and saves nothing (2048 tokens over
// 32768, bf16: heads of 128 1234 us so, 1223 exact; 64 399 : 409; 256 440 : 444).  Values likewise
// for fp16 outputs, and where not every row of a workgroup attends to all of a tile.  Elsewhere, for
// bf16, they are expanded to (c - z) scale 2^k, rounded to fp16: one step in 2^11 of a value, where
// a code of 8 bits is one in 2^8 of the row's largest and the output one in 2^8.  (Exact throughout
// they would cost heads of 64 another 14%, of 128 10%, of 256 6%.)
//
// The work is one line of tiles, shared out as in the step kernel.  A second kernel
// joins the partial results: a workgroup's has up to 133 KB, too much for the last
// one of an item to read them all.
//
// Measured: 2048 new tokens over 32768, 32/8 heads of 128, bf16, 1230 to 1290 us (0.82 to
// 0.86 PFLOP/s; a library product of 8192^3 reaches 1.14; the matrix units are busy in 40% of a
// SIMD's cycles, and other vector instructions take as many again); first chunks of 1500 to
// 4000 tokens, 16 heads of 64, fp16, 175 us, bf16 140; 9 chunks of up to 700 tokens, 16/4
// heads of 256, 4 bits, cap and window, 240 us, bound by issue with one wave on each SIMD.
#pragma once

#include "kvq_attention.h"

namespace onebit {

// Keys enter the products as (c - z) 2^-kKeyShift and their scales are held times
// 2^-kKeyScaleShift, so that a sum of 256 products (below 2^16) times any scale (below 2^122) stays
// below 2^127; the query row's factor makes up for both.  (That factor goes below fp32's
// smallest normal number only where max |q| * |sm_scale| is below 2^-138 and no score is above 1.)
constexpr int kKeyShift = 14, kKeyScaleShift = 12;
template <int BITS>
constexpr float kKeyUnit = (float)(1 << (kCodeShift<BITS> - kKeyShift));
constexpr int kChunkSeqs = 512;        // sequences of one launch
constexpr int kChunkMaxGroups = 1024;  // workgroups of one launch

// What workgroup w leaves for the join of the item that it begins and does not end.
struct ChunkSplit {
    int32_t last;  // the item's last workgroup; -1: there is no such item
    int32_t slot;  // of its first part
    int32_t q0;    // the sequence's first query
    int32_t row, rows;  // the item's first query row of the sequence, and how many
    int32_t head;
    int32_t pad[2];
};

template <int GT, int D, int NW>
struct ChunkPartial {
    float o[NW][D / 2][64];  // [wave][register][lane]
    float ml[NW][32][2];     // rows' maxima and sums
};

template <int GT, int D, int BITS, int NW>
struct ChunkShape {
    static constexpr int kThreads = 64 * NW, kRows = 32 * NW;
    static constexpr int kTile = D == 256 ? 32 : D == 128 ? 64 : 128;  // tokens
    // A thread expands 16 kWide key dimensions of a token and 4 kWide value dimensions of four.
    static constexpr int kWide = kTile * D / 16 / kThreads;
    static constexpr int kGroup = 4 * kWide;  // value dimensions of a thread
    static constexpr int kKeyRow = D + 8;                              // fp16 elements; 16 bytes of padding
    static constexpr int kValRow = kTile + 8;                          // spread the rows over the banks
    static constexpr int kCodeWords = BITS / 2;                        // words of 16 codes
    static constexpr int kValWords = BITS == 8 ? kWide : 1;            // words of a thread's codes of a value row
    static_assert(kWide * kThreads == kTile * D / 16 && (kWide == 1 || kWide == 2), "every thread expands whole pieces");
};

// N products whose left operands come from LDS, kAhead reads in front, with the pieces
// of some other work between them, in the order written: a product occupies the matrix
// cores for 32 cycles, in which the wave can issue the other work's instructions, but
// the compiler by itself puts every read right in front of its product and the other
// work behind them all.
constexpr int kAhead = 4;
// A value that a piece computes for later: the compiler would move its computation there.
__device__ __forceinline__ void pin(uint32_t &v) { asm volatile("" : "+v"(v)); }
// The largest of three, NaN if one is: one instruction, where fmaxf costs one more for
// each operand that might be a signalling NaN.  (A row with a NaN score comes out NaN
// whatever its running maximum.)
__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}
// The first reads are issued well before the products they feed.
template <int N, typename Read>
__device__ __forceinline__ void read_first(f16x8_v (&f)[kAhead], Read read) {
#pragma unroll
    for (int x = 0; x < kAhead && x < N; ++x) f[x] = read(x);
    __builtin_amdgcn_sched_barrier(0);
}
template <int N, int PIECES, typename Read, typename Product, typename Piece>
__device__ __forceinline__ void weave(f16x8_v (&f)[kAhead], Read read, Product product, Piece piece) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
#pragma unroll
        for (int x = p * N / PIECES; x < (p + 1) * N / PIECES; ++x) {
            product(x, f[x % kAhead]);
            if (x + kAhead < N) f[x % kAhead] = read(x + kAhead);
        }
        piece(p);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// 16 consecutive codes to fp16, in the order of query_operand
template <int BITS>
__device__ __forceinline__ void expand16(const uint32_t (&w)[BITS / 2], f16x2_v scale, f16x2_v offset, uint4 (&out)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const u32x4_v c = __builtin_bit_cast(
            u32x4_v, codes_over_dims<BITS>(w[BITS == 8 ? 2 * k : k], w[BITS == 8 ? 2 * k + 1 : k]));
        out[k] = make_uint4(fma16(c.x, scale, offset), fma16(c.y, scale, offset), fma16(c.z, scale, offset),
                            fma16(c.w, scale, offset));
    }
}

// Tiles of row tile `rt` of a sequence; base: the first tile's first token.
template <int ROWS, int TILE>
__host__ __device__ __forceinline__ int chunk_tiles(const KvqAttnArgs &a, const KvqSeq &s, int rt, int &base) {
    const int rows = s.len * a.group;
    const int t0 = rt * ROWS / a.group, t1 = (min(rows, (rt + 1) * ROWS) - 1) / a.group;
    base = kvq_lo(a, s, t0) & ~(TILE - 1);
    return max(1, (max(kvq_hi(s, t1) - base, 0) + TILE - 1) / TILE);
}

// What an item of a sequence is allotted in the line of work, in 1/16 tiles: its tiles
// (about) and what every item costs besides them, 8 us before its first tile, which is
// three tiles' time.  Row tile rt has first + rt * step, from row tile `grow` on, where
// windows are full, `full`.  Only the shares of the work depend on it; it need not be
// exact, but its sums have to be had at once.  (4000 new tokens under a window of 4096, 16
// heads of 64: 110 us with shares that do not grow, 95 so.)
struct ChunkShare {
    int64_t first, step, full;
    int32_t row_tiles, grow;
    __host__ __device__ __forceinline__ int64_t of(int rt) const { return rt < grow ? first + rt * step : full; }
    __host__ __device__ __forceinline__ int64_t before(int rt) const {
        const int64_t n = rt < grow ? rt : grow;
        return n * first + n * (n - 1) / 2 * step + (rt - n) * full;
    }
};
constexpr int kSetupTiles = 3;
template <int ROWS, int TILE>
__host__ __device__ __forceinline__ ChunkShare chunk_share(const KvqAttnArgs &a, const KvqSeq &s) {
    ChunkShare r{0, 0, 0, 0, 0};
    const int64_t rows = (int64_t)s.len * a.group;
    if (rows <= a.max_rows) return r;
    r.row_tiles = (int)((rows + ROWS - 1) / ROWS);
    const int tokens = (ROWS + a.group - 1) / a.group;  // of a row tile
    const int64_t reach = (s.kv > s.len ? s.kv - s.len : 0) + (int64_t)tokens;
    r.first = 16 * kSetupTiles + 16 * reach / TILE + 1;
    r.step = 16 * tokens >= TILE ? 16 * tokens / TILE : 1;
    r.grow = r.row_tiles;
    if (a.window > 0) {
        const int64_t most = (int64_t)a.window + tokens + TILE;
        const int64_t left = most > reach ? (most - reach + tokens - 1) / tokens : 0;
        if (left < r.grow) r.grow = (int)left;
        r.full = 16 * kSetupTiles + 16 * most / TILE + 1;
    }
    return r;
}

// A lane's outputs come in groups of four dimensions: register i_of of tile u_of holds
// dimension dim_of + k of the lane's row.
template <int D>
struct ChunkOut {
    static constexpr int kQuads = D / 8;
    static __device__ __forceinline__ constexpr int u_of(int q, int k) { return D == 64 ? k >> 1 : 4 * (q >> 4) + k; }
    static __device__ __forceinline__ constexpr int i_of(int q, int k) { return D == 64 ? q + 8 * (k & 1) : q & 15; }
    static __device__ __forceinline__ int dim_of(int q, int half) {
        return (D == 256 ? 8 : 4) * (8 * ((q & 15) >> 2) + 4 * half + (q & 3)) + 4 * (q >> 4);
    }
};

__device__ __forceinline__ int64_t out_row(const KvqAttnArgs &a, int q0, int g, int r) {
    return (int64_t)(q0 + r / a.group) * a.q_heads + g * a.group + r % a.group;
}
__device__ __forceinline__ float lse_of(float m, float l) {
    return l != 0.0f ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
}

template <int GT, int D, int BITS, int NW>
__global__ __launch_bounds__(64 * NW, NW / 4) void k_kvq_chunk(KvqAttnArgs a) {
    using S = ChunkShape<GT, D, BITS, NW>;
    constexpr bool kTwo = kTwoPart<GT>;  // weights in two parts, values exact; else scales fold into the values where they can
    constexpr int kTile = S::kTile, kWide = S::kWide, kMTiles = D / 32, kSteps = D / 16;
    // Where a weight by itself goes into the products (values folded), it is taken times 2^kWeightShift to
    // use fp16's range, and folded scales times 2^kFoldShift more than the row's exponent, so that both ways
    // add up to outputs in the same units.
    constexpr int kWeightShift = kTwo ? 0 : 7, kFoldShift = kCodeShift<BITS> - kUnitShift - kWeightShift;
    constexpr int kTopExp = 118;     // largest exponent of a row's values: 2^(kTopExp + kFoldShift) is a number
    constexpr int kByRow = 1 << 20;  // in place of a tile's exponent: each row has its own
    __shared__ _Float16 s_k[4][kTile][S::kKeyRow];
    __shared__ _Float16 s_v[4][D][S::kValRow];
    __shared__ float s_ks[4][kTile], s_vs[4][kTwo ? kTile : 1], s_log[4][kTile];
    __shared__ int64_t s_pre[kChunkSeqs + 1];
    __shared__ int64_t s_scan[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform((int)(tid >> 6));
    const int n = lane & 31, half = lane >> 5;

    ChunkSplit *splits = reinterpret_cast<ChunkSplit *>(static_cast<char *>(a.workspace));
    ChunkPartial<GT, D, NW> *parts =
        reinterpret_cast<ChunkPartial<GT, D, NW> *>(static_cast<char *>(a.workspace) + kChunkMaxGroups * sizeof(ChunkSplit));

    // ---- allotments of the sequences, as running sums
    {
        constexpr int kPer = (kChunkSeqs + S::kThreads - 1) / S::kThreads;
        int64_t u[kPer], sum = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int b = tid * kPer + k;
            u[k] = 0;
            if (b < a.batch) {
                const ChunkShare r = chunk_share<S::kRows, kTile>(a, kvq_seq(a, b));
                u[k] = r.before(r.row_tiles) * a.c.heads;
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
            if (tid * kPer + k < kChunkSeqs) s_pre[tid * kPer + k] = at;
            at += u[k];
        }
        if (tid == S::kThreads - 1) s_pre[kChunkSeqs] = at;
        __syncthreads();
    }
    const int64_t total = uniform(s_pre[kChunkSeqs]);
    // A stretch is allotted a tile at least, of the set-up's or the cache's.  (Small calls, against four tiles at least: 64 tokens over 1000 32 -> 25 us
    // with 8 heads of 64, 34 -> 31 us with heads of 128; the worst of 36 shapes 42 -> 43 us.)
    const int64_t groups = min((int64_t)gridDim.x, udiv(total + 15, 16));
    if (tid == 0) splits[blockIdx.x].last = -1;
    if ((int64_t)blockIdx.x >= groups) return;
    const int64_t each = udiv(total, groups), more = total - each * groups;
    const auto begin_of = [&](int64_t w) { return w * each + min(w, more); };
    const int64_t end = begin_of((int64_t)blockIdx.x + 1);
    int64_t pos = begin_of(blockIdx.x);
    int b;
    {
        int lo = 0, hi = kChunkSeqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] <= pos) lo = mid; else hi = mid;
        }
        b = uniform(lo);
    }

    for (bool first = true; pos < end; first = false) {
        while (s_pre[b + 1] <= pos) ++b;
        b = uniform(b);
        KvqSeq seq = kvq_seq(a, b);
        seq.q0 = uniform(seq.q0);
        seq.len = uniform(seq.len);
        seq.kv = uniform(seq.kv);
        const ChunkShare share = chunk_share<S::kRows, kTile>(a, seq);
        int64_t off = pos - uniform(s_pre[b]);
        int rt = 0;
        {
            int hi = share.row_tiles;  // before(rt) * heads <= off < before(hi) * heads
            while (hi - rt > 1) {
                const int mid = (rt + hi) >> 1;
                if (share.before(mid) * a.c.heads <= off) rt = mid; else hi = mid;
            }
            off -= share.before(rt) * a.c.heads;
        }
        int base;
        const int tiles = chunk_tiles<S::kRows, kTile>(a, seq, rt, base);
        const int64_t allotted = share.of(rt);
        const int g = uniform((int)udiv(off, allotted));
        const int64_t item_begin = pos - (off - g * allotted), item_end = item_begin + allotted;
        const int64_t seg_end = min(end, item_end);
        // the stretch's part of the item's tiles
        const int u0 = uniform((int)udiv((pos - item_begin) * tiles, allotted));
        const int u1 = uniform((int)udiv((seg_end - item_begin) * tiles, allotted));
        const int r0 = rt * S::kRows, r1 = min(seq.len * a.group, r0 + S::kRows);
        const int t0 = r0 / a.group, t1 = (r1 - 1) / a.group;
        const int some_hi = kvq_hi(seq, t1);                                  // attended to by some row of the tile
        const int every_lo = kvq_lo(a, seq, t1), every_hi = kvq_hi(seq, t0);  // ... by every row
        // (an item that attends to nothing reads nothing: the cache may have no pages)
        const int from = base + u0 * kTile, count = some_hi > base ? u1 - u0 : 0;
        const bool alone = pos == item_begin && seg_end == item_end;

        // ---- this lane's query row
        const int r = r0 + 32 * wave + n;
        const bool live = r < r1;
        const int my_t = live ? r / a.group : t1;
        const int my_lo = kvq_lo(a, seq, my_t), my_hi = kvq_hi(seq, my_t);
        const bool wave_live = r0 + 32 * wave < r1;  // (a wave without rows only expands)
        const int wt1 = (min(r1, r0 + 32 * wave + 32) - 1) / a.group;
        f16x8_v qf[kSteps];
        float qs;
        uint4 raw[kSteps];
        {
            const int h = live ? g * a.group + r % a.group : 0;
            const uint16_t *src = a.q + (int64_t)(seq.q0 + my_t) * a.q_token_stride + (int64_t)h * a.q_head_stride;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                raw[s] = live ? *reinterpret_cast<const uint4 *>(src + 16 * s + 8 * half) : make_uint4(0, 0, 0, 0);
        }
        const auto make_queries = [&]() {
            float amax = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    amax = fmaxf(amax, fmaxf(fabsf(half_bits_to_float<GT>(w[k] & 0xffffu)),
                                             fabsf(half_bits_to_float<GT>(w[k] >> 16))));
            }
            const int kq = query_exponent(fmaxf(amax, __shfl_xor(amax, 32, 64)));
            qs = ldexpf(a.scale2, kKeyShift + kKeyScaleShift - kq);
            // A factor of 0 goes into the queries: times the -inf of a key not attended to it would be NaN.
            const float up = qs == 0.0f ? 0.0f : __uint_as_float(__float_as_uint(pow2(kq)) ^ a.q_sign);
            qs = qs == 0.0f ? 1.0f : qs;
            if (a.cap2 > 0.0f) qs *= a.cap_scale;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
                float f[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = half_bits_to_float<GT>(w[k] & 0xffffu);
                    f[2 * k + 1] = half_bits_to_float<GT>(w[k] >> 16);
                }
                qf[s] = query_operand<BITS>(f, up);
            }
        };

        // ---- the tiles' way from the cache into LDS
        const int32_t *table = a.table + (int64_t)b * a.table_stride;
        // Page number of token j.  No branch, here or in row_of: the compiler would wait for
        // all loads under way where the ways join.  Tokens behind the table's end get its last page
        // (they are behind the sequence's end too, and so masked); a page outside the cache gives
        // rows of page 0, to be left out.
        const int last_page = (a.max_tokens >> a.c.shift) - 1;
        const uint32_t in_cache = (uint32_t)min(a.c.n_pages, (int64_t)1 << 31);
        const auto page_of = [&](int j) -> int { return table[min(j >> a.c.shift, last_page)]; };
        const auto there_is = [&](int page) { return (uint32_t)page < in_cache; };
        const auto row_of = [&](int page, int j) -> int64_t {
            return (int64_t)((((uint64_t)(uint32_t)(there_is(page) ? page : 0) * (uint32_t)a.c.heads + (uint32_t)g)
                              << a.c.shift) |
                             (uint32_t)(j & (a.c.page - 1)));
        };
        // A wave's threads expand consecutive tokens of one page, the same for keys and values.
        constexpr int kRowBytes = D * BITS / 8, kGroup = S::kGroup;
        const int first_token = wave * (1024 * kWide / D);
        const int k_token = lane / (D / 16 / kWide), k_dim = 16 * kWide * (lane % (D / 16 / kWide));
        const int v_token = 4 * (lane / (D / kGroup)), v_dim = kGroup * (lane % (D / kGroup));
        // tokens of the tile that a lane watches the scales of (two rounds for 128 tokens)
        constexpr int kWatch = kTile > 64 ? 2 : 1;
        struct Pages {
            int piece, watch[kWatch];
        };
        struct Stage {
            uint32_t kw[kWide][S::kCodeWords], vw[4][S::kValWords];
            float ks, kv;  // both scales of the key row
            float4 vs;
            int page;
            float w_vs[kWatch];
            bool w_there[kWatch];
        };
        uint64_t there_next[kWatch];  // tokens whose pages are in the cache
        const auto watch_token = [&](int i) { return (64 * i + lane) % kTile; };
        const auto load_pages = [&](Pages &p, int j) {
            p.piece = page_of(j + first_token);
#pragma unroll
            for (int i = 0; i < kWatch; ++i) p.watch[i] = page_of(j + watch_token(i));
        };
        const auto load_tile = [&](Stage &s, const Pages &p, int j) {
            s.page = uniform(p.piece);
            const int64_t row = row_of(s.page, j + first_token);
            const float *ksp = a.c.scales[0] + row, *vsp = a.c.scales[1] + row;
            s.ks = ksp[k_token];
            s.kv = vsp[k_token];
            s.vs = *reinterpret_cast<const float4 *>(vsp + v_token);
            const uint32_t *kp = reinterpret_cast<const uint32_t *>(a.c.codes[0] + row * kRowBytes + k_token * kRowBytes +
                                                                    k_dim * BITS / 8);
            // (words of codes, as many at a time as a load takes)
            constexpr int kKeyWords = kWide * S::kCodeWords;
            uint32_t *kw = &s.kw[0][0];
            if (kKeyWords == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(kp);
                kw[0] = v.x; kw[1] = v.y;
            } else {
#pragma unroll
                for (int t = 0; t < kKeyWords; t += 4) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(kp + t);
                    kw[t] = v.x; kw[t + 1] = v.y; kw[t + 2] = v.z; kw[t + 3] = v.w;
                }
            }
            const uint8_t *vp = a.c.codes[1] + row * kRowBytes + v_token * kRowBytes + v_dim * BITS / 8;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint8_t *q = vp + t * kRowBytes;
                if (S::kValWords == 2) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(q);
                    s.vw[t][0] = v.x;
                    s.vw[t][S::kValWords - 1] = v.y;
                } else {
                    s.vw[t][0] = kGroup * BITS / 8 == 4 ? *reinterpret_cast<const uint32_t *>(q)
                                                        : *reinterpret_cast<const uint16_t *>(q);
                }
            }
#pragma unroll
            for (int i = 0; i < kWatch; ++i) {
                const int at = j + watch_token(i);
                const int64_t wr = row_of(p.watch[i], at);
                s.w_vs[i] = a.c.scales[1][wr];
                s.w_there[i] = there_is(p.watch[i]);
            }
        };
        Pages pages, pages0, pages1;
        Stage stage;
        if (count > 0) {
            load_pages(pages0, from);
            load_pages(pages1, from + kTile);
        }
        // Value scales are brought into fp16's range by a power of two, chosen for the largest that a
        // row attends to, itself: other rows' tokens must not decide what is lost of its values.  Where
        // every row attends to all of a tile the largest is common to them, and its exponent is the
        // tile's; elsewhere (the diagonal, the front of a window) scales go to the weights in fp32, by their
        // logarithms in s_log.
        float v_top = 0.0f;                       // the largest of the former tiles so far
        int v_exp_top = kTopExp, v_exp_next = 0;  // its exponent; that of the tile being expanded
        float x_ks, x_vs, x_s4[4];                // what becomes of its scales
        const auto expand_begin = [&](const Stage &s, int buf, int j) {
            const bool every = j >= every_lo && j + kTile <= every_hi;
            float vt = 0.0f;
            bool plain = every;
#pragma unroll
            for (int i = 0; i < kWatch; ++i) {
                const float y = fabsf(s.w_vs[i]);
                const bool in = s.w_there[i] && y < INFINITY;
                there_next[i] = __ballot(s.w_there[i]);
                plain = plain && __ballot(in) == ~0ull;
                vt = fmaxf(vt, in ? y : 0.0f);
            }
            if (__builtin_expect(every && __any(vt > v_top), 0)) {
#pragma unroll
                for (int d = 32; d >= 1; d >>= 1) vt = fmaxf(vt, __shfl_xor(vt, d, 64));
                v_top = fmaxf(v_top, vt);
                v_exp_top = uniform(min(value_exponent(v_top), kTopExp));
            }
            v_exp_next = every ? v_exp_top : kByRow;
            const float vf = pow2(v_exp_top + (kTwo ? 0 : kFoldShift)), v4[4] = {s.vs.x, s.vs.y, s.vs.z, s.vs.w};
            x_ks = fmaf(s.ks, 0.0f, s.ks) * pow2(-kKeyScaleShift);  // (NaN for an infinite scale)
            x_vs = s.kv * vf;
#pragma unroll
            for (int t = 0; t < 4; ++t) x_s4[t] = v4[t] * vf;
            if (__builtin_expect(!plain, 0)) {
                // A scale that is not finite makes the scores of its token NaN and its values 0: NaN for the
                // rows that attend to it, nothing for the others.
                const bool ok = there_is(s.page), finite = fabsf(s.kv) < INFINITY;
                x_ks = finite ? x_ks : NAN;
                x_vs = !every ? copysignf(1.0f, s.kv) : ok && finite ? x_vs : 0.0f;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    x_s4[t] = !every ? copysignf(kUnitScale<BITS>, v4[t]) : ok && fabsf(v4[t]) < INFINITY ? x_s4[t] : 0.0f;
                if (!every && k_dim == 0)
                    s_log[buf][first_token + k_token] = ok && finite ? log2f(fabsf(s.kv)) : -INFINITY;
            }
        };
        // the expansion in pieces: 16 key dimensions, then a dimension of the values at a time
        constexpr int kPieces = 5 * kWide;
        const auto expand_piece = [&](const Stage &s, int buf, int piece) {
            if (piece < kWide) {
                uint4 x[2];
                expand16<BITS>(s.kw[piece], splat16(kKeyUnit<BITS>), splat16(-0x1p-17f * kKeyUnit<BITS>), x);
                uint4 *dst = reinterpret_cast<uint4 *>(&s_k[buf][first_token + k_token][k_dim + 16 * piece]);
                dst[0] = x[0];
                dst[1] = x[1];
                if (k_dim == 0 && piece == 0) {
                    s_ks[buf][first_token + k_token] = x_ks;
                    if (kTwo) s_vs[buf][first_token + k_token] = x_vs;
                }
            } else {
                const int d = piece - kWide, w = BITS == 8 ? d / 4 : 0;
                f16x2_v s2[2];
#pragma unroll
                for (int t = 0; t < 4; ++t) s2[t >> 1][t & 1] = (_Float16)(kTwo ? kUnitScale<BITS> : x_s4[t]);
                // four tokens are eight bytes; of each 16 tokens, those that one half of a wave
                // multiplies lie together
                const int quad = (first_token + v_token) / 4;
                const int to = 16 * (quad / 4) + 8 * (quad & 1) + 4 * ((quad >> 1) & 1);
                const uint32_t lo = fma16(code_pair<BITS>(s.vw[0][w], s.vw[1][w], d), s2[0], s2[0] * (_Float16)-0x1p-17f);
                const uint32_t hi = fma16(code_pair<BITS>(s.vw[2][w], s.vw[3][w], d), s2[1], s2[1] * (_Float16)-0x1p-17f);
                *reinterpret_cast<uint2 *>(&s_v[buf][d * (D / kGroup) + v_dim / kGroup][to]) = make_uint2(lo, hi);
            }
        };

        constexpr int kSubs = kTile / 32, kPv = 2 * kMTiles;
        f32x16_v o[kMTiles], acc[2];  // outputs; scores of this step and the next
        u32x4_v pw[2][2], lw[2][2];   // weights of this step and the last, each for two products of 16 tokens
        float m = kNone, l = 0.0f;
        float f_grow = 1.0f, scale = 0.0f, shift = 0.0f, l_keep = 0.0f;
        bool grow = false, by_row = false;
        int v_exp = kTopExp;                   // the row's: of what its outputs have summed
        int l_exp = 0;                         // l is 2^(l_exp + kWeightShift) times the sum of the weights
        int v_exps[3];                         // of tiles it, it + 1, it + 2
        uint64_t theres[2][kWatch];            // of tiles it, it + 1
#pragma unroll
        for (int u = 0; u < kMTiles; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[u][i] = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) pw[t][k] = lw[t][k] = (u32x4_v){0u, 0u, 0u, 0u};
        const auto read_k = [&](int buf, int sub, int x) {
            return *reinterpret_cast<const f16x8_v *>(&s_k[buf][32 * sub + n][16 * x + 8 * half]);
        };
        const auto read_v = [&](int buf, int sub, int x) {
            return *reinterpret_cast<const f16x8_v *>(
                &s_v[buf][32 * (x % kMTiles) + n][32 * sub + 16 * (x / kMTiles) + 8 * half]);
        };
        const auto mul_k = [&](f32x16_v &to, int x, f16x8_v f) {
            to = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, qf[x], to, 0, 0, 0);
        };
        const auto mul_v = [&](int w, int x, f16x8_v f) {
            const int u = x % kMTiles, t = x / kMTiles;
            o[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, __builtin_bit_cast(f16x8_v, pw[w][t]), o[u], 0, 0, 0);
            if (kTwo)
                o[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, __builtin_bit_cast(f16x8_v, lw[w][t]), o[u], 0, 0, 0);
        };
        const auto clear = [](f32x16_v &x) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.0f;
        };
        // scores of step `sub` of the tile in `buf`, whose first token is js: scale, cap and mask, and the
        // row's running maximum and exponent.  `top` is the row's largest raw score where that is all
        // there is to do; `other`: the tile's exponent is not the last one's.  A row's numbers depend on its
        // own tokens only.  (Branches are marked as rare where most steps pass them by: laid out in line
        // they cost 2048 tokens over 32768 8%.)
        const auto settle = [&](f32x16_v &x, float top, int buf, int sub, int js, int t_exp, bool other, const uint64_t (&here2)[kWatch]) {
            const uint32_t here = (uint32_t)(here2[sub / 2] >> (32 * (sub & 1)));
            uint32_t mine = ~0u;  // the tokens that this lane's row attends to, one bit each, from its half's first
            by_row = t_exp == kByRow;
            scale = qs;
            if (__builtin_expect(a.cap2 > 0.0f || by_row || here != ~0u, 0)) {
                if (a.cap2 > kWideCap2) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = capped_wide(x[i] * qs, a.cap2);
                    scale = 1.0f;
                } else if (a.cap2 > 0.0f) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = capped(x[i] * qs, a.cap2);
                    scale = 1.0f;
                }
                if (by_row || here != ~0u) {
                    const int lo = min(max(my_lo - js, 0), 32), hi = min(max(my_hi - js, 0), 32);
                    const uint64_t bits = ((1ull << hi) - 1) & ~((1ull << lo) - 1) & here;
                    mine = (uint32_t)(bits >> (4 * half));
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!(mine >> (8 * (i / 4) + (i & 3)) & 1)) x[i] = -INFINITY;
                }
                top = x[0];
#pragma unroll
                for (int i = 0; i < 16; i += 2) top = max3(top, x[i], x[i + 1]);
            }
            f_grow = 1.0f;
            grow = false;
            if (__builtin_expect(other && !by_row, 0)) {
                // In a tile with an exponent of its own the weights are short of the row's units by the
                // difference, and l with them.  (2^-90 of a weight is nothing in fp16, while l has room for it.)
                const int e = min(v_exp, t_exp), le = max(e - t_exp, -90);
                grow = __any(e != v_exp);
                f_grow = ldexpf(1.0f, e - v_exp);
                l = ldexpf(l, le - l_exp);
                v_exp = e;
                l_exp = le;
            }
            if (__builtin_expect(__any(top * scale > m + 8.0f), 0)) {
                grow = true;
                top = fmaxf(top, __shfl_xor(top, 32, 64)) * scale;
                const bool up = top > m + 8.0f;
                const float f = up ? exp2_fast(m - top) : 1.0f;
                m = up ? top : m;
                l *= f;
                f_grow *= f;
            }
            shift = (float)(kWeightShift + l_exp) - m;
            if (__builtin_expect(by_row, 0)) {
                // The logarithms of weight times scale are computed here, with the power of two that brings the
                // row's largest below 2^15 (they are 2^-18 off), and the weights' sum, so that the loop below
                // knows nothing of it; it adds up something else for l, which is put right after it.
                l_keep = l;
                if (__any(mine != 0)) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(&s_log[buf][32 * sub + 2 * i + 4 * half]);
                        const float v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float w = fmaf(x[i + k], scale, -m);
                            sum += exp2_fast(w);
                            x[i + k] = w + v4[k];
                        }
                    }
                    float most = x[0];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) most = max3(most, x[i], x[i + 1]);
                    most = fmaxf(most, __shfl_xor(most, 32, 64));
                    const int e = most > -INFINITY ? min(v_exp, 14 - (int)floorf(most)) : v_exp;
                    grow |= __any(e != v_exp);
                    f_grow = ldexpf(f_grow, e - v_exp);
                    v_exp = e;
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] += (float)e;
                    l_keep += ldexpf(sum, kWeightShift + l_exp);
                }
                scale = 1.0f;
                shift = 0.0f;
            }
        };
        // the key scales, applied to the scores in fp32
        const auto scale_keys = [&](f32x16_v &x, int buf, int sub, int i) {
            const float4 f = *reinterpret_cast<const float4 *>(&s_ks[buf][32 * sub + 2 * i + 4 * half]);
            x[i] *= f.x; x[i + 1] *= f.y; x[i + 2] *= f.z; x[i + 3] *= f.w;
        };

        if (count > 0) {
            // two tiles in LDS and the third on its way.  (Loads past the last tile are of rows that
            // exist; what is made of them is not used.)
            Stage second;
            load_tile(stage, pages0, from);
            load_tile(second, pages1, from + kTile);
            load_pages(pages, from + 2 * kTile);
            make_queries();
            __syncthreads();  // the item before is done with the buffers
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                expand_begin(t ? second : stage, t, from + t * kTile);
#pragma unroll
                for (int x = 0; x < kPieces; ++x) expand_piece(t ? second : stage, t, x);
                v_exps[t] = v_exp_next;
#pragma unroll
                for (int i = 0; i < kWatch; ++i) theres[t][i] = there_next[i];
                if (t == 0) {
                    load_tile(stage, pages, from + 2 * kTile);
                    load_pages(pages, from + 3 * kTile);
                }
            }
            __syncthreads();
            if (wave_live) {
                clear(acc[0]);
#pragma unroll
                for (int x = 0; x < kSteps; ++x) mul_k(acc[0], x, read_k(0, 0, x));
#pragma unroll
                for (int i = 0; i < 16; i += 4) scale_keys(acc[0], 0, 0, i);
                float top = acc[0][0];
#pragma unroll
                for (int i = 0; i < 16; i += 2) top = max3(top, acc[0][i], acc[0][i + 1]);
                settle(acc[0], top, 0, 0, from, v_exps[0], true, theres[0]);
            }
        }
        const auto load_next = [&](int j) {
            const Pages p = pages;
            load_pages(pages, j + 4 * kTile);
            load_tile(stage, p, j + 3 * kTile);
        };
        // A step is 32 tokens.  While its weights are computed, the matrix cores multiply the next
        // step's scores and the last step's values; in a tile's first step the tile after next is
        // expanded, too.  Four tiles' places in LDS: the one before this, whose last values are
        // still to be multiplied, this and the next one, and the one being expanded.
        // The last values of a wave, of tile `it`.  (No maximum has moved since their weights were computed.)
        const auto last_values = [&](int it) {
#pragma unroll
            for (int x = 0; x < kPv; ++x) mul_v(kSubs == 1 ? 1 : (kSubs - 1) & 1, x, read_v(it & 3, kSubs - 1, x));
        };
        // (a wave whose rows attend to nothing further on only expands: above a diagonal of 256 tokens)
        const int wave_hi = wave_live ? kvq_hi(seq, wt1) : 0;
        bool working = wave_live;
        for (int it = 0; it < count; ++it) {
            const int j = from + it * kTile, buf = it & 3, after = (it + 1) & 3, fresh = (it + 2) & 3;
            if (it > 0) __syncthreads();
            if (working && it > 0 && j >= wave_hi) {
                last_values(it - 1);
                working = false;
            }
            if (!working) {
                expand_begin(stage, fresh, j + 2 * kTile);
#pragma unroll
                for (int x = 0; x < kPieces; ++x) expand_piece(stage, fresh, x);
                load_next(j);
                continue;
            }
#pragma unroll
            for (int sub = 0; sub < kSubs; ++sub) {
                const int cur = kSubs == 1 ? 0 : sub & 1, nxt = cur ^ 1;
                const bool wrap = sub + 1 == kSubs;  // the next step is the next tile's first
                const int kb = wrap ? after : buf, ks = wrap ? 0 : sub + 1;
                // (before the first step there are no last values: weights of 0, and any finite values)
                const int vb = sub ? buf : it ? (it - 1) & 3 : 0, vs = sub ? sub - 1 : kSubs - 1;
                constexpr int kN = kSteps + kPv;
                const auto read = [&](int x) { return x < kSteps ? read_k(kb, ks, x) : read_v(vb, vs, x - kSteps); };
                f16x8_v ahead[kAhead];
                read_first<kN>(ahead, read);
                if (sub == 0) {
                    expand_begin(stage, fresh, j + 2 * kTile);
                    v_exps[2] = v_exp_next;
                }
                f32x16_v &x = acc[cur], &y = acc[nxt];
                clear(y);
                const auto weigh = [&](int q) {  // of two tokens, relative to the running maximum
                    const int i = 2 * q;
                    float e[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) e[k] = exp2_fast(fmaf(x[i + k], scale, shift));
                    l += e[0] + e[1];
                    if (kTwo) {
                        const float2 v = *reinterpret_cast<const float2 *>(
                            &s_vs[buf][32 * sub + 8 * (i / 4) + 4 * half + (i & 3)]);
                        e[0] *= v.x;
                        e[1] *= v.y;
                    }
                    uint32_t p = round_pair<kGradF16>(e[0], e[1]), rest = 0;
                    if (kTwo) {
                        rest = rest_pair(e[0], e[1], p);
                        pin(rest);
                        lw[cur][i / 8][(i % 8) / 2] = rest;
                    }
                    pin(p);
                    pw[cur][i / 8][(i % 8) / 2] = p;
                };
                float top = kNone;
                const auto largest = [&](int i) {  // of four of the next scores
                    scale_keys(y, kb, ks, i);
                    top = max3(max3(top, y[i], y[i + 1]), y[i + 2], y[i + 3]);
                };
                constexpr int kFirst = kPieces + 1;  // pieces of a tile's first step more than of the others
                const auto piece = [&](int p) {
                    if (sub > 0) p += kFirst;
                    if (p < kPieces)
                        expand_piece(stage, fresh, p);
                    else if (p < kFirst)
                        load_next(j);
                    else if (p < kFirst + 8)
                        weigh(p - kFirst);
                    else
                        largest(4 * (p - kFirst - 8));
                };
                const auto product = [&](int x, f16x8_v g) { if (x < kSteps) mul_k(y, x, g); else mul_v(nxt, x - kSteps, g); };
                if (sub == 0)
                    weave<kN, kFirst + 12>(ahead, read, product, piece);
                else
                    weave<kN, 12>(ahead, read, product, piece);
                if (__builtin_expect(by_row, 0)) l = l_keep;
                // (the last values went in with weights relative to the maximum and the exponent before this step's)
                if (__builtin_expect(grow, 0)) {
#pragma unroll
                    for (int u = 0; u < kMTiles; ++u)
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[u][i] *= f_grow;
                }
                const bool other = wrap && v_exps[1] != v_exps[0];
                if (wrap) {
                    v_exps[0] = v_exps[1];
                    v_exps[1] = v_exps[2];
#pragma unroll
                    for (int i = 0; i < kWatch; ++i) {
                        theres[0][i] = theres[1][i];
                        theres[1][i] = there_next[i];
                    }
                }
                grow = false;
                if (!wrap || it + 1 < count)
                    settle(y, top, kb, ks, wrap ? j + kTile : j + 32 * (sub + 1), v_exps[0], other, theres[0]);
                if (kSubs == 1) {
                    x = y;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        pw[1][k] = pw[0][k];
                        lw[1][k] = lw[0][k];
                    }
                }
            }
        }
        if (count > 0 && working) last_values(count - 1);

        // ---- results
        l += __shfl_xor(l, 32, 64);
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        l = ldexpf(l, -kWeightShift - l_exp);
#pragma unroll
        for (int u = 0; u < kMTiles; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[u][i] = ldexpf(o[u][i] * inv, kUnitShift + kWeightShift + l_exp - v_exp);
        if (alone) {
            if (live) {
                using O = ChunkOut<D>;
                const int64_t to = out_row(a, seq.q0, g, r);
#pragma unroll
                for (int q = 0; q < O::kQuads; ++q) {
                    const float v[4] = {o[O::u_of(q, 0)][O::i_of(q, 0)], o[O::u_of(q, 1)][O::i_of(q, 1)],
                                        o[O::u_of(q, 2)][O::i_of(q, 2)], o[O::u_of(q, 3)][O::i_of(q, 3)]};
                    store_out4<GT>(a.out + to * D + O::dim_of(q, half), v);
                }
                if (a.lse && half == 0) a.lse[to] = lse_of(m, l);
            }
        } else {
            const int slot = 2 * blockIdx.x + (first ? 0 : 1);
            if (wave_live) {
#pragma unroll
                for (int u = 0; u < kMTiles; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) parts[slot].o[wave][16 * u + i][lane] = o[u][i];
                if (half == 0) {
                    parts[slot].ml[wave][n][0] = m;
                    parts[slot].ml[wave][n][1] = l;
                }
            }
            if (tid == 0 && pos == item_begin) {
                const int64_t at = more * (each + 1), unit = item_end - 1;
                ChunkSplit s{};
                s.last = (int)(unit < at ? udiv(unit, each + 1) : more + udiv(unit - at, each));
                s.slot = slot;
                s.q0 = seq.q0;
                s.row = r0;
                s.rows = r1 - r0;
                s.head = g;
                splits[blockIdx.x] = s;
            }
        }
        pos = seg_end;
    }
}

// Joins the parts of the items that a workgroup of k_kvq_chunk, of `groups`, began and
// did not end.  A task is the rows of one of that workgroup's waves; each of four waves
// here takes a quarter of their dimensions.  Where there are few such items, of many
// parts each (long caches), a task is one quarter, and of that the four waves take every
// fourth part each: a wave by itself would wait for one after the other.  The first wave
// adds up their sums, in their order.  The workgroups share the tasks out between them:
// one for every task that there might be would take longer to start and end the idle
// ones than the others take to work.  Measured with 8 heads of 128: 8 us where one
// sequence of 48 rows has 32 parts an item (24 us by one wave for each quarter), 17.6 us
// where items have two full parts (67 MB, 14 us at the rate of a copy).
constexpr int kJoinWaves = 4;
template <int GT, int D, int NW>
__global__ __launch_bounds__(64 * kJoinWaves) void k_kvq_chunk_join(KvqAttnArgs a, int groups) {
    using O = ChunkOut<D>;
    constexpr int kMine = O::kQuads / 4, kBatch = 2, kPer = kChunkMaxGroups / (64 * kJoinWaves);
    __shared__ float s_v[kJoinWaves - 1][4 * kMine][64], s_ml[kJoinWaves - 1][64][2];
    __shared__ int16_t s_items[kChunkMaxGroups];
    __shared__ int s_count[kJoinWaves];
    const ChunkSplit *splits = reinterpret_cast<const ChunkSplit *>(a.workspace);
    const ChunkPartial<GT, D, NW> *parts = reinterpret_cast<const ChunkPartial<GT, D, NW> *>(
        static_cast<const char *>(a.workspace) + kChunkMaxGroups * sizeof(ChunkSplit));
    const int lane = threadIdx.x & 63, line = uniform((int)(threadIdx.x >> 6));
    const int n = lane & 31, half = lane >> 5;

    // the workgroups that began such an item
    uint64_t has[kPer];
    int count = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int w = 64 * (kPer * line + k) + lane;
        has[k] = __ballot(w < groups && splits[min(w, groups - 1)].last >= 0);
        count += __popcll(has[k]);
    }
    if (lane == 0) s_count[line] = count;
    __syncthreads();
    int items = 0, at = 0;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) {
        at += w < line ? s_count[w] : 0;
        items += s_count[w];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (has[k] >> lane & 1) s_items[at + __popcll(has[k] & ((1ull << lane) - 1))] = (int16_t)(64 * (kPer * line + k) + lane);
        at += __popcll(has[k]);
    }

    items = uniform(items);
    const int lines = 4 * items < groups ? kJoinWaves : 1, tasks = items * NW * lines;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        __syncthreads();  // s_items is written; the task before is done with the sums
        const int at = task / lines, begin = uniform((int)s_items[at / NW]), wave = at % NW;
        const int quarter = lines > 1 ? task % lines : line;
        const ChunkSplit s = splits[begin];
        if (32 * wave >= s.rows) continue;
        float v[kMine][4], m = kNone, l = 0.0f;
#pragma unroll
        for (int q = 0; q < kMine; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[q][k] = 0.0f;
        const auto add = [&](const float (&o)[kMine][4], float pm, float pl) {
            const float top = fmaxf(m, pm), f0 = exp2_fast(m - top), f = pl * exp2_fast(pm - top);
            m = top;
            l = l * f0 + f;
#pragma unroll
            for (int q = 0; q < kMine; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[q][k] = fmaf(o[q][k], f, v[q][k] * f0);
        };
        for (int w = begin + (lines > 1 ? line : 0); w <= s.last; w += kBatch * lines) {
            float o[kBatch][kMine][4], pm[kBatch], pl[kBatch];
#pragma unroll
            for (int t = 0; t < kBatch; ++t) {
                // (past the last part the one at w again, with nothing of it)
                const int at = w + t * lines <= s.last ? w + t * lines : w;
                const ChunkPartial<GT, D, NW> &p = parts[at == begin ? s.slot : 2 * at];
                pm[t] = p.ml[wave][n][0];
                pl[t] = t == 0 || at != w ? p.ml[wave][n][1] : 0.0f;
#pragma unroll
                for (int q = 0; q < kMine; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // the register's number, with `quarter` the only part that is not a constant
                        const int x = kMine * quarter + q;
                        o[t][q][k] = p.o[wave][16 * O::u_of(x, k) + O::i_of(x, k)][lane];
                    }
            }
#pragma unroll
            for (int t = 0; t < kBatch; ++t) add(o[t], pm[t], pl[t]);
        }
        if (lines > 1) {
            if (line > 0) {
#pragma unroll
                for (int q = 0; q < kMine; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s_v[line - 1][4 * q + k][lane] = v[q][k];
                s_ml[line - 1][lane][0] = m;
                s_ml[line - 1][lane][1] = l;
            }
            __syncthreads();
            if (line > 0) continue;
            // (a wave's sums are not divided by l: they enter with the weight 1)
#pragma unroll
            for (int w = 0; w < kJoinWaves - 1; ++w) {
                const float pm = s_ml[w][lane][0], top = fmaxf(m, pm), f0 = exp2_fast(m - top), f = exp2_fast(pm - top);
                m = top;
                l = l * f0 + s_ml[w][lane][1] * f;
#pragma unroll
                for (int q = 0; q < kMine; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[q][k] = fmaf(s_v[w][4 * q + k][lane], f, v[q][k] * f0);
            }
        }
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        if (32 * wave + n < s.rows) {
            const int64_t to = out_row(a, s.q0, s.head, s.row + 32 * wave + n);
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const float x[4] = {v[q][0] * inv, v[q][1] * inv, v[q][2] * inv, v[q][3] * inv};
                store_out4<GT>(a.out + to * D + O::dim_of(kMine * quarter + q, half), x);
            }
            if (a.lse && quarter == 0 && half == 0) a.lse[to] = lse_of(m, l);
        }
    }
}

}  // namespace onebit
