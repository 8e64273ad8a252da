// Attention of the newest tokens of each sequence over a paged cache held in 4 bits.
//
// Query m of a sequence of length n sits at position p = n - M + m and sees the tokens max(0, p + 1 - window) .. p
// (window 0: all): out = sum_t softmax_t(scale q . k_t) v_t. The queries that share a key head (group * M rows) read
// each of its cached rows once.
//
// Arithmetic. Both products run on m16n8k16 matrix instructions over the codes themselves: a 4-bit code at bits 0-3 of a
// half ORed with the pattern of 1024 is 1024 + code, at bits 4-7 it is 1024 + 16 code, and one packed subtraction leaves
// code - 8 or 16 (code - 8), exactly; the factor 16 is folded into q (scores) or into the output element (values). (The
// bare codes as f16 subnormals need no subtraction, but the matrix unit aligns its products by the operands' unnormalised
// exponents and keeps 7 bits less: scores 2^-17 off instead of 2^-24.) A block's scale multiplies the fp32 sum of its 32
// products (keys) or the softmax weight (values), so what is rounded to f16 is only
//   - q, scaled to the row's largest magnitude: exact for f16 and bf16 queries, and for fp32 queries split into a high
//     and a low f16 part (22 bits) that fill the two halves of the instruction's 16 rows;
//   - the weight times its value scale, kept within 2^15 by the running reference below: one f16 for 16-bit outputs
//     (half a step 2^-12), a high and a low part for fp32.
// Scores, running maximum, running sum and outputs are fp32. The reference that the exponentials subtract is the row's
// running maximum plus the exponent of the largest value scale so far, so weight * scale never leaves f16's range.
//
// Work. A warp takes tiles of 32 tokens, streamed by cp.async into its own ring of shared-memory stages (16-byte chunks
// XOR-swizzled so that ldmatrix is free of bank conflicts; ldmatrix delivers the keys' words in the layout of a column
// operand, and ldmatrix.trans the values' half-words with two tokens in one register, which is what a row operand along
// tokens wants). All tiles of a call, (sequence, key head, group of rows) by (sequence, ...), are divided evenly over
// the resident CTAs, whatever the lengths; a CTA joins its warps through shared memory and writes the output of what it
// holds whole, and a second kernel joins what was divided between CTAs, always in the same order.
#include "kv_common.cuh"

namespace q4 {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;      // tokens a warp takes at a time
constexpr int kMaxB = 1024;    // sequences of a call
constexpr int kStages = 3;     // tiles of a warp in flight or in use
constexpr int kItemCost = 6;   // what starting on an item costs a CTA, in tiles

template <int DB>
struct Geo {
    static constexpr int D = DB * 32;
    static constexpr int kRow = DB * 16;                   // code bytes of a cache row
    static constexpr int kCodes = kTile * kRow;            // of a tile
    static constexpr int kScales = kTile * DB * 2;
    static constexpr int kStage = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
    static constexpr int kCtas = DB == 8 ? 2 : 3;          // CTAs per SM
    static constexpr int kJoinRow = D + 4;                 // floats; the pad spreads the joining stores over the banks
};

struct Params {
    KvAttnArgs a;
    float* part;  // [G][2][8 NT * (D + 2)]
    int4* desc;   // [G]: the item that begins in a CTA and ends in a later one: (sequence, head * chunks + chunk, last CTA, slot)
    int R, group, chunks, lp;  // rows per key head, query heads per key head, chunks of 8 NT rows, log2(page size)
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// 16, 8 or 4 bytes global -> shared, zeros instead where `bytes` is 0.
template <int SIZE>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t bytes) {
    if constexpr (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(SIZE), "r"(bytes) : "memory");
}

template <int WORDS>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(addr + 4u * i)
                         : "memory");
    }
}

// A row's 16-byte chunk c sits at chunk c ^ swizzle(row), so that eight rows of one chunk cover all banks.
template <int DB>
__device__ __forceinline__ int swizzled(int row, int c) {
    return c ^ ((row * DB / 8) & (DB - 1));
}

// What a sequence's length means: tokens [lo, n) are read, in tiles from `first` on.
struct Span {
    int n, lo, first, tiles;
    bool bad;
};
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, int len) {
    Span s;
    s.bad = len < 0 || len > a.max_pages * a.c.page_size;
    s.n = s.bad ? 0 : len;
    s.lo = a.window > 0 ? max(0, s.n - a.M + 1 - a.window) : 0;
    s.first = s.lo & ~(kTile - 1);
    s.tiles = max(1, (s.n - s.first + kTile - 1) / kTile);  // an empty sequence's zeros are somebody's to write
    return s;
}

// prefix[b] = cost (of one key head and chunk) of the sequences before b, prefix[B] = of all. An item costs its tiles and
// kItemCost for its start: 64 ragged sequences with empty and one-token ones among them took 168 us where tiles alone
// were divided (the CTA with all the short ones worked alone for 60 us).
__device__ void scan_tiles(const KvAttnArgs& a, long long* prefix) {
    __shared__ long long warp_sum[kWarps];
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = threadIdx.x * per;
    long long sum = 0;
    for (int b = b0; b < min(a.B, b0 + per); ++b) sum += span_of(a, a.seq_lens[b]).tiles + kItemCost;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
    }
    if (lane == 31) warp_sum[warp] = up;
    __syncthreads();
    long long at = up - sum;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    for (int b = b0; b < min(a.B, b0 + per); ++b) {
        prefix[b] = at;
        at += span_of(a, a.seq_lens[b]).tiles + kItemCost;
        if (b == a.B - 1) prefix[a.B] = at;
    }
    __syncthreads();
}

__device__ __forceinline__ float2 to_float2(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

// Eight codes of a word (four of each half, from bit 0 up) as f16 pairs: code - 8 (pairs 0, 2) and 16 (code - 8) (1, 3).
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t (&x)[4]) {
    const uint32_t w8 = w >> 8;
    x[0] = (w & 0x000F000Fu) | 0x64006400u;
    x[1] = (w & 0x00F000F0u) | 0x64006400u;
    x[2] = (w8 & 0x000F000Fu) | 0x64006400u;
    x[3] = (w8 & 0x00F000F0u) | 0x64006400u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t off = i % 2 ? 0x64806480u : 0x64086408u;  // 1152, 1032
        __half2 a, b;
        memcpy(&a, &x[i], 4);
        memcpy(&b, &off, 4);
        a = __hsub2(a, b);
        memcpy(&x[i], &a, 4);
    }
}

// Four query elements.
__device__ __forceinline__ void load_q4(const void* q, long long at, int dtype, float (&x)[4]) {
    if (dtype == Q4_F32) {
        load_floats(static_cast<const float*>(q) + at, x);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at);
        const float2 lo = dtype == Q4_F16 ? unpack2(w.x, __half()) : unpack2(w.x, __nv_bfloat16());
        const float2 hi = dtype == Q4_F16 ? unpack2(w.y, __half()) : unpack2(w.y, __nv_bfloat16());
        x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
    }
}

__device__ __forceinline__ void store_out4(const KvAttnArgs& a, long long at, float4 v) {
    if (a.dtype == Q4_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
    else if (a.dtype == Q4_F16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack2(v.x, v.y, __half()), pack2(v.z, v.w, __half()));
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
            make_uint2(pack2(v.x, v.y, __nv_bfloat16()), pack2(v.z, v.w, __nv_bfloat16()));
}

// Row r of a key head's rows: query r / group, query head h * group + r % group. Its place in out, and in lse.
__device__ __forceinline__ long long out_at(const Params& p, int b, int h, int r, int D) {
    return ((long long)b * p.a.M + r / p.group) * p.a.out_stride + (long long)(h * p.group + r % p.group) * D;
}
__device__ __forceinline__ long long lse_at(const Params& p, int b, int h, int r) {
    return ((long long)b * p.a.M + r / p.group) * p.a.Hq + h * p.group + r % p.group;
}
// lse from the reference (a power of two) and the sum under it.
__device__ __forceinline__ float lse_of(float ref, float l) {
    return l == 0.f ? -INFINITY : 0.69314718055994531f * (ref + log2f(l));
}

// SPLIT: fp32 queries and outputs, high and low parts. NT: groups of 8 rows that a CTA holds at once.
template <int DB, int NT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, Geo<DB>::kCtas) kv4_attention_kernel(const Params p) {
    using G = Geo<DB>;
    constexpr int D = G::D, MT = SPLIT ? NT : (NT + 1) / 2, ROWS = 8 * NT;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ long long prefix[kMaxB + 1];
    __shared__ float join_ref[kWarps][ROWS], join_l[kWarps][ROWS];
    const KvAttnArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const uint32_t base = smem_addr(ring) + (uint32_t)(warp * kStages * G::kStage);

    grid_dependency_wait();
    grid_launch_dependents();
    scan_tiles(a, prefix);
    const int items = a.c.num_kv_heads * p.chunks;
    const long long total = prefix[a.B] * items;
    // an even share of the cost, no less than an item of one tile per warp
    const long long share = max((total + gridDim.x - 1) / (long long)gridDim.x, (long long)(kWarps + kItemCost));
    const long long begin = min(total, share * blockIdx.x), end = min(total, begin + share);
    if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);

    for (long long at = begin; at < end;) {
        // the item (sequence b, head h, chunk) that place `at` belongs to, and how many of its tiles are this CTA's
        int b = 0;
        for (int step = 512; step > 0; step >>= 1)
            if (b + step < a.B && prefix[b + step] * items <= at) b += step;
        const Span s = span_of(a, a.seq_lens[b]);
        const long long rem = at - prefix[b] * items;
        const int cost = s.tiles + kItemCost;
        const int item = (int)(rem / cost), from = (int)(rem - (long long)item * cost);  // tiles follow the item's start
        const int tile0 = max(from - kItemCost, 0);
        const int count = (int)min(end - at + from - kItemCost, (long long)s.tiles) - tile0;
        const long long item_at = at - from;
        at = min(end, item_at + cost);
        if (count <= 0) break;  // the share ends in the item's start: its tiles are the next CTA's
        const int h = item / p.chunks, row0 = (item - h * p.chunks) * ROWS;
        const int* table = a.block_table + (long long)b * a.max_pages;
        bool bad = s.bad;

        // the cache row of this lane's token of the warp's i-th tile, -1 where none is read
        auto lookup = [&](int i) {
            const int t = s.first + (tile0 + i * kWarps + warp) * kTile + lane;
            if (i * kWarps + warp >= count || t < s.lo || t >= s.n) return -1;
            const int page = table[t >> p.lp];
            if (page < 0 || page >= a.c.num_pages) return -2;
            return (int)cache_row(a.c, page, h, t & (a.c.page_size - 1));
        };
        // lane's part of a tile's copies: chunk `lane % DB` of every (32 / DB)-th token, and the scales of token `lane`
        const uint8_t *k_src = a.c.k_qs + (lane % DB) * 16, *v_src = a.c.v_qs + (lane % DB) * 16;
        auto issue = [&](int i, int row) {
            if (i * kWarps + warp < count) {
                const uint32_t st = base + (uint32_t)(i % kStages) * G::kStage;
                const uint32_t ds = st + 2 * G::kCodes + (uint32_t)(lane * DB * 2);
                auto copies = [&](auto all) {  // all: every token of the tile is read
                    constexpr bool ALL = decltype(all)::value;
#pragma unroll
                    for (int j = 0; j < DB; ++j) {
                        const int tok = (j * 32 + lane) / DB;
                        const int r = __shfl_sync(0xffffffffu, row, tok);
                        const long long off = (long long)(ALL ? r : max(r, 0)) * G::kRow;
                        const uint32_t dst = st + (uint32_t)(tok * G::kRow + swizzled<DB>(tok, lane % DB) * 16);
                        const uint32_t bytes = ALL || r >= 0 ? 16u : 0u;
                        copy_async<16>(dst, k_src + off, bytes);
                        copy_async<16>(dst + G::kCodes, v_src + off, bytes);
                    }
                    const long long off = (long long)(ALL ? row : max(row, 0)) * DB;
                    const uint32_t bytes = ALL || row >= 0 ? DB * 2 : 0;
                    copy_async<DB * 2>(ds, a.c.k_d + off, bytes);
                    copy_async<DB * 2>(ds + G::kScales, a.c.v_d + off, bytes);
                };
                if (__all_sync(0xffffffffu, row >= 0)) {
                    copies(std::true_type());
                } else {
                    if (row == -2) bad = true;
                    copies(std::false_type());
                }
            }
            cp_async_commit();
        };
        int rows_ahead[kStages];
#pragma unroll
        for (int i = 0; i < kStages; ++i) rows_ahead[i] = lookup(i);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(i, rows_ahead[i]);
        int row_next = rows_ahead[kStages - 1];

        // queries: scaled so that the row's largest lies in [2^13, 2^14), split, in the layout of the row operand
        uint32_t qa[MT][DB][2][4];
        float factor[NT];      // row g: score * log2(e) = factor * accumulated sum
        int seen_end[NT], seen_lo[NT];
#pragma unroll
        for (int i = 0; i < MT * DB * 2 * 4; ++i) (&qa[0][0][0][0])[i] = 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + n * 8 + g;
            const bool there = r < p.R;
            float x[DB][8];
            float top = 0.f;
            bool finite = true;
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                float u[4] = {}, v[4] = {};
                if (there) {
                    const long long at_q = ((long long)b * a.M + r / p.group) * a.q_stride +
                                           (long long)(h * p.group + r % p.group) * D + 32 * k + 4 * t4;
                    load_q4(a.q, at_q, a.dtype, u);
                    load_q4(a.q, at_q + 16, a.dtype, v);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[k][j] = u[j], x[k][4 + j] = v[j];
                    finite = finite && fabsf(u[j]) < INFINITY && fabsf(v[j]) < INFINITY;
                    top = fmaxf(top, fmaxf(fabsf(u[j]), fabsf(v[j])));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const unsigned quad = __ballot_sync(0xffffffffu, finite) >> (lane & ~3) & 15u;
            // largest in [2^(e), 2^(e+1)): scale by 2^(13 - e), as two factors that stay in range
            const int e = max((int)(__float_as_uint(top) >> 23), 1) - 127;
            const int k2 = top > 0.f && quad == 15u ? 13 - e : 0;
            const float f1 = pow2i(k2 / 2), f2 = pow2i(k2 - k2 / 2);
            factor[n] = quad == 15u ? (a.scale * 1.4426950408889634f) * pow2i(-(k2 / 2)) * pow2i(-(k2 - k2 / 2)) : qnan();
            const int m = r / p.group;
            seen_end[n] = there ? s.n - a.M + m + 1 : 0;
            seen_lo[n] = a.window > 0 ? seen_end[n] - a.window : 0;
            const int mt = SPLIT ? n : n / 2, hi = SPLIT ? 0 : n % 2;
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                float xh[8], xl[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float y = quad == 15u ? (x[k][j] * f1) * f2 : 0.f;
                    if (j >= 4) y *= 0.0625f;
                    xh[j] = __half2float(__float2half_rn(y));
                    xl[j] = __half2float(__float2half_rn(y - xh[j]));
                }
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    qa[mt][k][o][hi] = pack_half2(xh[o], xh[o + 2]);
                    qa[mt][k][o][2 + hi] = pack_half2(xh[4 + o], xh[6 + o]);
                }
                if constexpr (SPLIT) {
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        qa[mt][k][o][1] = pack_half2(xl[o], xl[o + 2]);
                        qa[mt][k][o][3] = pack_half2(xl[4 + o], xl[6 + o]);
                    }
                }
            }
        }
        // tokens that every row of this chunk sees, so that only tiles outside it look at each token
        const int last_row = min(p.R, row0 + ROWS) - 1;
        const int all_end = s.n - a.M + row0 / p.group + 1;
        const int all_lo = a.window > 0 ? s.n - a.M + last_row / p.group + 1 - a.window : 0;

        float o[NT][DB][2][4];      // element 2g + j (c0, c1) and 16 + 2g + j (c2, c3) of rows 2 t4, 2 t4 + 1
        float top[NT], ref[NT], l[NT];  // row g: running maximum, reference, the lane's part of the sum
#pragma unroll
        for (int i = 0; i < NT * DB * 8; ++i) (&o[0][0][0][0])[i] = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) top[n] = -INFINITY, ref[n] = 0.f, l[n] = 0.f;
        int e_run = -14;

#pragma unroll 1
        for (int i = 0; i * kWarps + warp < count; ++i) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            issue(i + kStages - 1, row_next);
            row_next = lookup(i + kStages);
            const uint32_t st = base + (uint32_t)(i % kStages) * G::kStage;
            const int tok0 = s.first + (tile0 + i * kWarps + warp) * kTile;

            auto tile = [&](auto masked) {
            constexpr bool MASKED = decltype(masked)::value;  // some row does not see every token
            // scores: sc[n][j] of row g, tokens 8 (j / 2) + 2 t4 + j % 2
            float sc[NT][8];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 8; ++j) sc[n][j] = 0.f;
            uint32_t kd[4][DB];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                lds_words<DB>(st + 2 * G::kCodes + (uint32_t)((8 * j + 2 * t4) * DB * 2), kd[j]);
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                uint32_t w[4];
                ldsm4(st + (uint32_t)(lane * G::kRow + swizzled<DB>(lane, k) * 16), w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 da = to_float2(kd[j][k / 2]), db = to_float2(kd[j][DB / 2 + k / 2]);
                    const float2 d = make_float2(k % 2 ? da.y : da.x, k % 2 ? db.y : db.x);
                    uint32_t x[4];
                    codes_of(w[j], x);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                        float c[4];
                        mma(c, qa[mt][k][0], x[0], x[1], zero);
                        mma(c, qa[mt][k][1], x[2], x[3], c);
                        if constexpr (SPLIT) {
                            const float2 both = fadd2(make_float2(c[0], c[1]), make_float2(c[2], c[3]));
                            const float2 y = ffma2(both, d, make_float2(sc[mt][2 * j], sc[mt][2 * j + 1]));
                            sc[mt][2 * j] = y.x, sc[mt][2 * j + 1] = y.y;
                        } else {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int n = 2 * mt + u;
                                if (n < NT) {
                                    const float2 y = ffma2(make_float2(c[2 * u], c[2 * u + 1]), d,
                                                           make_float2(sc[n][2 * j], sc[n][2 * j + 1]));
                                    sc[n][2 * j] = y.x, sc[n][2 * j + 1] = y.y;
                                }
                            }
                        }
                    }
                }
            }

            // the largest exponent of a value scale, so far (zeros stand where nothing was read)
            {
                uint32_t own[DB / 2], m = 0u;
                if constexpr (DB == 2) own[0] = lds32(st + 2 * G::kCodes + G::kScales + (uint32_t)(lane * 4));
                else lds_words<DB / 2>(st + 2 * G::kCodes + G::kScales + (uint32_t)(lane * DB * 2), own);
#pragma unroll
                for (int k = 0; k < DB / 2; ++k) m = max(m, max(own[k] & 0x7C00u, (own[k] >> 16) & 0x7C00u));
                e_run = max(e_run, (int)(__reduce_max_sync(0xffffffffu, m) >> 10) - 15);
            }
            bool moved = false;
            float keep[NT];
            uint32_t seen[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                seen[n] = 0u;
                if constexpr (MASKED) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int t = tok0 + 8 * (j / 2) + 2 * t4 + j % 2;
                        if (t >= seen_lo[n] && t < seen_end[n]) seen[n] |= 1u << j;
                        else sc[n][j] = -INFINITY;
                    }
                }
                float m = sc[n][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) m = fmaxf(m, sc[n][j]);
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const float nt = fmaxf(top[n], m * factor[n]);
                const float nr = (nt == -INFINITY ? 0.f : nt) + (float)(e_run - 14);
                keep[n] = top[n] == -INFINITY ? 1.f : ex2(ref[n] - nr);  // nothing to keep before the first token
                moved = moved || nr != ref[n];
                top[n] = nt;
                ref[n] = nr;
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    l[n] *= keep[n];
                    const float ka = __shfl_sync(0xffffffffu, keep[n], 8 * t4);
                    const float kb = __shfl_sync(0xffffffffu, keep[n], 8 * t4 + 4);
#pragma unroll
                    for (int k = 0; k < DB; ++k) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) o[n][k][j][0] *= ka, o[n][k][j][1] *= kb, o[n][k][j][2] *= ka, o[n][k][j][3] *= kb;
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sc[n][j] = ex2(fmaf(sc[n][j], factor[n], -ref[n]));
                    if (MASKED && !(seen[n] >> j & 1u)) sc[n][j] = 0.f;  // also where the query is not finite
                    l[n] += sc[n][j];
                }
            }

            uint32_t vd[4][DB];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                lds_words<DB>(st + 2 * G::kCodes + G::kScales + (uint32_t)((8 * j + 2 * t4) * DB * 2), vd[j]);
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                uint32_t w[4];
                ldsm4_trans(st + G::kCodes + (uint32_t)(lane * G::kRow + swizzled<DB>(lane, k) * 16), w);
                uint32_t hi[NT][4], lo[NT][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 da = to_float2(vd[j][k / 2]), db = to_float2(vd[j][DB / 2 + k / 2]);
                    const float2 d = make_float2(k % 2 ? da.y : da.x, k % 2 ? db.y : db.x);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float2 y = __fmul2_rn(make_float2(sc[n][2 * j], sc[n][2 * j + 1]), d);
                        if constexpr (MASKED) {  // a masked token's scale may be anything
                            if (!(seen[n] >> (2 * j) & 1u)) y.x = 0.f;
                            if (!(seen[n] >> (2 * j + 1) & 1u)) y.y = 0.f;
                        }
                        hi[n][j] = pack_half2(y.x, y.y);
                        if constexpr (SPLIT) {
                            const float2 back = to_float2(hi[n][j]);
                            lo[n][j] = pack_half2(y.x - back.x, y.y - back.y);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t x[4], y[4];
                    codes_of(w[2 * u], x);
                    codes_of(w[2 * u + 1], y);
                    const uint32_t a0[4] = {x[0], x[1], y[0], y[1]}, a1[4] = {x[2], x[3], y[2], y[3]};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma(o[n][k][0], a0, hi[n][2 * u], hi[n][2 * u + 1], o[n][k][0]);
                        mma(o[n][k][1], a1, hi[n][2 * u], hi[n][2 * u + 1], o[n][k][1]);
                        if constexpr (SPLIT) {
                            mma(o[n][k][0], a0, lo[n][2 * u], lo[n][2 * u + 1], o[n][k][0]);
                            mma(o[n][k][1], a1, lo[n][2 * u], lo[n][2 * u + 1], o[n][k][1]);
                        }
                    }
                }
            }
            };
            if (tok0 >= all_lo && tok0 >= s.lo && tok0 + kTile <= all_end) tile(std::false_type());
            else tile(std::true_type());
        }
        cp_async_wait<0>();
        bad = __any_sync(0xffffffffu, bad) != 0;
        __syncthreads();  // every warp's stages are free: the join uses their memory

        float* jo = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
            if (t4 == 0) {
                join_l[warp][8 * n + g] = bad ? qnan() : l[n];
                join_ref[warp][8 * n + g] = bad ? 0.f : l[n] == 0.f ? -INFINITY : ref[n];
            }
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                float* to = jo + (size_t)(warp * ROWS + 8 * n + 2 * t4) * G::kJoinRow + 32 * k + 2 * g;
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // elements 2g + j, and 16 + 2g + j with their factor of 16 more
                    const float f = half ? 0.0625f : 1.f;
                    const float2 x = make_float2(o[n][k][0][2 * half] * f, o[n][k][1][2 * half] * f);
                    const float2 y = make_float2(o[n][k][0][2 * half + 1] * f, o[n][k][1][2 * half + 1] * f);
                    *reinterpret_cast<float2*>(to + 16 * half) = x;
                    *reinterpret_cast<float2*>(to + G::kJoinRow + 16 * half) = y;
                }
            }
        }
        if (bad && lane == 0) atomicOr(a.fault, s.bad ? (unsigned)kFaultBadLength : (unsigned)kFaultBadPage);
        __syncthreads();
        const bool whole = count == s.tiles;
        const int slot = item_at + kItemCost <= begin ? 0 : 1;  // an item that began before is this CTA's first
        float* part = p.part + ((long long)blockIdx.x * 2 + slot) * (ROWS * (D + 2));
        for (int idx = threadIdx.x; idx < ROWS * (D / 4); idx += kThreads) {
            const int r = idx / (D / 4), d4 = idx % (D / 4);
            if (row0 + r >= p.R) continue;
            float rt = -INFINITY, lt = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) rt = fmaxf(rt, join_ref[w][r]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (rt != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (join_ref[w][r] == -INFINITY) continue;  // saw nothing
                    const float f = ex2(join_ref[w][r] - rt);
                    const float4 x = *reinterpret_cast<const float4*>(jo + (size_t)(w * ROWS + r) * G::kJoinRow + 4 * d4);
                    lt = fmaf(join_l[w][r], f, lt);
                    v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
                }
            }
            if (whole) {
                const float inv = lt == 0.f ? 0.f : 1.f / lt;
                store_out4(a, out_at(p, b, h, row0 + r, D) + 4 * d4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                if (a.lse && d4 == 0) a.lse[lse_at(p, b, h, row0 + r)] = lse_of(rt, lt);
            } else {
                *reinterpret_cast<float4*>(part + r * D + 4 * d4) = v;
                if (d4 == 0) part[ROWS * D + r] = rt, part[ROWS * D + ROWS + r] = lt;
            }
        }
        if (threadIdx.x == 0 && tile0 == 0 && !whole) {
            // the item begins here: a join starts from this CTA
            p.desc[blockIdx.x] = make_int4(b, item, (int)((item_at + cost - 1) / share), slot);
        }
        __syncthreads();  // the join's memory is free for the next stages
    }
}

// Joins the parts of the items that were divided between CTAs: block (c, r) row r of the item that begins in CTA c.
template <int DB, int NT>
__global__ void __launch_bounds__(256) kv4_attention_join_kernel(const Params p) {
    constexpr int D = DB * 32, ROWS = 8 * NT, kJoinWarps = 8;
    __shared__ float so[kJoinWarps][D], sl[kJoinWarps], sm[kJoinWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int4 ds = p.desc[blockIdx.x];
    if (ds.x < 0) return;
    const int r = blockIdx.y, h = ds.y / p.chunks, row = (ds.y - h * p.chunks) * ROWS + r;
    if (row >= p.R) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x, n = ds.z - c0 + 1;
    auto part = [&](int i) { return p.part + ((long long)(c0 + i) * 2 + (i == 0 ? ds.w : 0)) * (ROWS * (D + 2)); };
    float top = -INFINITY;
    for (int i = threadIdx.x; i < n; i += 256) top = fmaxf(top, part(i)[ROWS * D + r]);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (lane == 0) sm[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sm[w]);
    float v[DB] = {}, l = 0.f;
    if (top != -INFINITY) {
#pragma unroll 4
        for (int i = warp; i < n; i += kJoinWarps) {
            const float* x = part(i);
            const float ref = x[ROWS * D + r];
            const float f = ex2(ref - top);  // 0 for a part that saw nothing (ref -infinity)
            l = fmaf(x[ROWS * D + ROWS + r], f, l);
#pragma unroll
            for (int k = 0; k < DB; ++k) v[k] = fmaf(x[r * D + 32 * k + lane], f, v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < DB; ++k) so[warp][32 * k + lane] = v[k];
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    float lt = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) lt += sl[w];
    for (int d4 = threadIdx.x; d4 < D / 4; d4 += 256) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&so[w][4 * d4]);
            t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
        }
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        store_out4(p.a, out_at(p, ds.x, h, row, D) + 4 * d4, make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv));
        if (p.a.lse && d4 == 0) p.a.lse[lse_at(p, ds.x, h, row)] = lse_of(top, lt);
    }
}

// Groups of 8 rows that a CTA holds: two where there are more than 8 rows and the outputs fit the registers.
int row_groups(int M, int group, int D) { return M * group > 8 && D < 256 ? 2 : 1; }

template <typename F>
auto with_plan(int D, int nt, bool split, F fn) {
    auto by_split = [&](auto db, auto n) {
        return split ? fn(db, n, std::true_type()) : fn(db, n, std::false_type());
    };
    using one = std::integral_constant<int, 1>;
    using two = std::integral_constant<int, 2>;
    if (D == 64) return nt == 2 ? by_split(two(), two()) : by_split(two(), one());
    if (D == 128) return nt == 2 ? by_split(std::integral_constant<int, 4>(), two()) : by_split(std::integral_constant<int, 4>(), one());
    return by_split(std::integral_constant<int, 8>(), one());
}

}  // namespace

size_t kv4_attention_workspace_bytes(int M, int group, int D, int dtype, int sm_count) {
    const int nt = row_groups(M, group, D);
    return with_plan(D, nt, dtype == Q4_F32, [&](auto db, auto n, auto) {
        constexpr int DB = decltype(db)::value, NT = decltype(n)::value;
        const size_t ctas = (size_t)sm_count * Geo<DB>::kCtas;
        return ctas * (sizeof(int4) + 2 * 8 * NT * (DB * 32 + 2) * sizeof(float));
    });
}

cudaError_t launch_kv4_attention(const KvAttnArgs& a, void* workspace, int sm_count, cudaStream_t s) {
    const int group = a.Hq / a.c.num_kv_heads, nt = row_groups(a.M, group, a.c.head_dim);
    return with_plan(a.c.head_dim, nt, a.dtype == Q4_F32, [&](auto db, auto n, auto split) {
        constexpr int DB = decltype(db)::value, NT = decltype(n)::value;
        auto kernel = kv4_attention_kernel<DB, NT, decltype(split)::value>;
        constexpr int kRing = kWarps * kStages * Geo<DB>::kStage;
        static_assert(kRing >= kWarps * 8 * NT * Geo<DB>::kJoinRow * 4, "the join must fit in the ring");
        static_assert((DB != 8 || NT == 1), "more rows than registers");
        const int ctas = sm_count * Geo<DB>::kCtas;
        Params p;
        p.a = a;
        p.desc = static_cast<int4*>(workspace);
        p.part = reinterpret_cast<float*>(p.desc + ctas);
        p.R = group * a.M;
        p.group = group;
        p.chunks = (p.R + 8 * NT - 1) / (8 * NT);
        p.lp = 0;
        while ((1 << p.lp) < a.c.page_size) ++p.lp;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
        if (e == cudaSuccess) e = launch_grid(kernel, dim3((unsigned)ctas), dim3(kThreads), kRing, s, launch_overlap(), p);
        // the join starts as soon as the main kernel's writes are there, whatever the overlap setting: it is this call's own
        if (e == cudaSuccess)
            e = launch_grid(kv4_attention_join_kernel<DB, NT>, dim3((unsigned)ctas, 8 * NT), dim3(256), 0, s, true, p);
        return e;
    });
}

}  // namespace q4
