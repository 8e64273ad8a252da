// Attention of the newest tokens of each sequence over a paged cache held in 4 bits.
//
// Query m of a sequence of length n sits at position p = n - M + m and sees the tokens max(0, p + 1 - window) .. p
// (window 0: all): out = sum_t softmax_t(scale q . k_t) v_t. The queries that share a key head (group * M rows) read
// and decode each of its cached rows once for every 16 of them (8 at head size 256).
//
// Arithmetic. Both products run on m16n8k16 matrix instructions over the codes themselves: a 4-bit code at bits 0-3 of a
// half ORed with the pattern of 1024 is 1024 + code, at bits 4-7 it is 1024 + 16 code, and one packed subtraction leaves
// code - 8 or 16 (code - 8), exactly; the factor 16 is folded into q (scores) or into the output element (values). (The
// bare codes as f16 subnormals need no subtraction, but the matrix unit aligns its products by the operands' unnormalised
// exponents and keeps 7 bits less: scores 2^-17 off instead of 2^-24.) A block's scale multiplies the fp32 sum of its 32
// products (keys) or the softmax weight (values), so what is rounded to f16 is only
//   - q, scaled to the row's largest magnitude: f16 and bf16 queries as they are, fp32 queries split into a high and a low
//     f16 part (22 bits) that fill the two halves of the instruction's 16 rows. Elements far below the largest meet f16's last
//     step and are off by up to 2^-34 of the largest, which a score's own roundings exceed unless a token's key scales differ
//     by more than 2^14;
//   - the weight times its value scale, a term: one f16 for 16-bit outputs (half a step: 2^-11 of it), a high and a low part
//     (2^-22) for fp32.
// Scores, running maximum, running sum and outputs are fp32. The reference that the exponentials subtract is the row's
// running maximum plus the exponent of the largest value scale so far, so that the largest terms lie below 2^15. Scales that
// differ by up to 2^10 leave the row's largest term in every block at 2^4 or above; what f16 loses below its step of 2^-24
// is then, over n tokens, at most n 2^-29 of it, less than the roundings of an fp32 sum of n. A row that has seen scales
// further apart (or some zeros; and every row in a tile of which the rows of a warp see different tokens) is `apart`: its
// terms are scaled by the tile's own largest one in each block. Tokens that a row does not see change none of its bits.
//
// Work. A warp takes tiles of 32 tokens, streamed by cp.async into its own ring of shared-memory stages (16-byte chunks
// XOR-swizzled so that ldmatrix is free of bank conflicts; ldmatrix delivers the keys' words in the layout of a column
// operand, and ldmatrix.trans the values' half-words with two tokens in one register, which is what a row operand along
// tokens wants). An item is a sequence, a key head and a chunk of 8 NT of its query rows. Two ways to divide the items:
//   - streams: all items' tiles lie on one line, which is cut into a piece of equal cost for each resident warp, whatever
//     the lengths. A warp walks its piece without meeting another warp, its copies running ahead across items; it writes
//     the outputs of items that it holds whole, and parts of the others, which a second kernel joins in a fixed order.
//   - whole items: one CTA per item, its warps' tiles interleaved and joined through shared memory; one launch.
#include <algorithm>
#include <atomic>
#include <cfloat>

#include "kv_common.cuh"

namespace q4 {

namespace {

constexpr int kTile = 32;       // tokens a warp takes at a time
constexpr int kMaxB = 1024;     // sequences of a call
constexpr int kItemCost = 4;    // what starting on an item costs a streaming warp, in tiles
// A row is `apart` once the value scales that it has seen differ by more than 2^kRange, or some block had zeros and others (a
// block that is zero throughout, as in padded heads, has nothing to lose). 64 ragged sequences (bf16, heads of 128): 71 us,
// 77 us with a block of zeros, 113 us with a zero scale among others in every page.
constexpr int kRange = 10, kNone = -100;
constexpr uint32_t kNoneSeen = 16u + 64u;  // Rows::e_own before the first token

template <int DB>
struct Geo {
    static constexpr int D = DB * 32;
    static constexpr int kRow = DB * 16;                   // code bytes of a cache row
    static constexpr int kCodes = kTile * kRow;            // of a tile
    static constexpr int kScales = kTile * DB * 2;
    static constexpr int kStage = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
    static constexpr int kJoinRow = D + 4;                 // floats; the pad spreads the joining stores over the banks
};

// Warps and stages (tiles of a warp in flight or in use), by registers and shared memory: on an SM 8 warps of up to 255
// registers, 12 of 168 or 16 of 128.
template <int DB, int NT, bool SPLIT>
struct Plan {  // streams
    static constexpr bool kSixteen = DB == 4 && NT == 1 && !SPLIT, kTwelve = DB == 2 || (DB == 4 && NT == 1);
    static constexpr int kWarps = kSixteen ? 16 : kTwelve ? 12 : 8;  // warps of an SM, all in one CTA
    static constexpr int kStages = kSixteen ? 2 : DB == 2 ? 5 : DB == 4 && NT == 1 ? 3 : DB == 4 ? 4 : 2;
};
enum : int { kFew, kMany, kCrowd };  // CTAs of an items launch
template <int DB, int NT, bool SPLIT, int COUNT>
struct ItemPlan {  // items: CTAs that hide each other's starts, or few; a crowd has one start a warp less
    static constexpr bool kSix = COUNT == kFew && DB <= 4 && NT == 1 && !SPLIT;
    static constexpr int kWarps = COUNT == kCrowd ? 2 : kSix ? 6 : 4;        // warps of a CTA
    static constexpr int kCtas = COUNT == kFew ? 2 : COUNT == kMany ? 4 : 8;  // CTAs of an SM
    static constexpr int kStages = COUNT != kFew ? (DB == 2 ? 4 : 2) : DB == 8 ? 2 : kSix ? 3 : 4;
};

struct Params {
    KvAttnArgs a;
    float* part;  // [warps][2][8 NT * (D + 2)]
    int2* desc;   // [B * items]: the parts of an item (1: it was whole), the first one's warp * 2 + slot
    int R, group, chunks, lp;  // rows per key head, query heads per key head, chunks of 8 NT rows, log2(page size)
    int warps;                 // streaming warps; 0: whole or split items
    int splits;                // CTAs of an item
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

__device__ __forceinline__ void lds_floats(uint32_t addr, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x[i]), "=f"(x[i + 1]), "=f"(x[i + 2]), "=f"(x[i + 3])
                     : "r"(addr + 4u * i)
                     : "memory");
}
__device__ __forceinline__ void lds_floats4(uint32_t addr, float (&x)[4]) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(addr) : "memory");
}
// An 8 x 8 matrix of halves, a row's pair of columns in each lane, transposed.
__device__ __forceinline__ uint32_t turned_over(uint32_t w) {
    uint32_t x;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(x) : "r"(w));
    return x;
}
__device__ __forceinline__ void sts_word(uint32_t addr, uint32_t w) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(w) : "memory");
}
__device__ __forceinline__ void sts_quad(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
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

// A token's scales: one, two or four words.
template <int WORDS>
__device__ __forceinline__ void lds_own(uint32_t addr, uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
    else lds_words<WORDS>(addr, w);
}

// Token t of a tile lies in row place(t) of its stage; lane l of an ldmatrix gives the address of row l % 8 of matrix l / 8,
// which is row row_of_lane(l).
//   Tokens along columns: column c of matrix j is token 8 (c / 2) + 2 j + c % 2, so that a lane's eight tokens (columns
//   2 t4 and 2 t4 + 1 of four matrices) are the consecutive ones 8 t4 .. 8 t4 + 7.
//   Tokens along rows (KT): row i of matrix j is token 4 i + j, a lane's four tokens are 4 g .. 4 g + 3. (The exclusive or
//   spreads the neighbours that a copy instruction writes over the banks.)
template <bool KT>
__device__ __forceinline__ int place(int t) {
    return KT ? 8 * (t & 3) + ((t >> 2) ^ (t & 3)) : 8 * (t >> 1 & 3) + 2 * (t >> 3) + (t & 1);
}
template <bool KT>
__device__ __forceinline__ int row_of_lane(int lane) {
    return KT ? lane ^ (lane >> 3) : lane;
}

// A row's 16-byte chunk c sits at chunk c ^ swizzle(row), so that eight rows of one chunk cover all banks.
template <int DB>
__device__ __forceinline__ int swizzle(int row) {
    return (row * DB / 8) & (DB - 1);
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

// (w & mask) | or_: one instruction, with `or_` in a register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t or_) {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "n"(MASK), "r"(or_));
    return x;
}
// Eight codes of a word (four of each half, from bit 0 up) as f16 pairs: code - 8 (pairs 0, 2) and 16 (code - 8) (1, 3).
// `k1024`: 1024 in both halves, in a register that the compiler does not know the value of (it would set it anew at
// every use).
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t k1024, uint32_t (&x)[4]) {
    const uint32_t w8 = w >> 8;
    x[0] = and_or<0x000F000Fu>(w, k1024);
    x[1] = and_or<0x00F000F0u>(w, k1024);
    x[2] = and_or<0x000F000Fu>(w8, k1024);
    x[3] = and_or<0x00F000F0u>(w8, k1024);
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


__device__ __forceinline__ uint32_t half_max(uint32_t a, uint32_t b) {
    uint32_t x;
    asm("max.f16x2 %0, %1, %2;" : "=r"(x) : "r"(a), "r"(b));
    return x;
}
__device__ __forceinline__ uint32_t half_min(uint32_t a, uint32_t b) {
    uint32_t x;
    asm("min.f16x2 %0, %1, %2;" : "=r"(x) : "r"(a), "r"(b));
    return x;
}

// One warp's state on an item. SPLIT: fp32 queries and outputs, high and low parts. NT: groups of 8 query rows.
//
// Queries that fill the 16 rows of an instruction (two groups of 16-bit ones, the two parts of fp32 ones) are its row
// operand and the keys its columns, and the scores lie as the values' instruction wants the weights. A single group of
// 16-bit queries would fill half of it; there (KT) the keys are the rows and the 8 queries the columns, half as many
// instructions and fewer registers, and movmatrix turns the weights over (64 ragged sequences 74 us with the queries as
// rows, 70 us so and with 16 warps; one of 131001 tokens 41 and 38 us; both sides before rows could be apart).
template <int DB, int NT, bool SPLIT>
struct Rows {
    using G = Geo<DB>;
    static constexpr bool KT = !SPLIT && NT == 1;
    static constexpr int D = G::D, MT = SPLIT ? NT : (NT + 1) / 2, ROWS = 8 * NT;
    static constexpr int LR = KT ? 2 : NT;  // rows whose softmax a lane has a part in: row g of each group; KT: 2 t4, 2 t4 + 1
    int lane, g, t4;
    uint32_t k1024;             // see codes_of
    uint32_t queries;           // shared address of this lane's operands: [MT][DB][2] of 16 bytes (KT: 8), kQuad apart
    float factor[LR];           // of a row: score * log2(e) = factor * accumulated sum
    int seen_end[LR], seen_lo[LR];  // a row sees the tokens seen_lo .. seen_end - 1
    int all_end, all_lo;        // tokens that every row sees, so that only tiles outside look at each token
    float o[NT][DB][2][4];      // element 2g + j (c0, c1) and 16 + 2g + j (c2, c3; 16-fold) of rows 2 t4, 2 t4 + 1
    float top[LR], l[LR];       // of a row: running maximum, the lane's part of the sum
    bool same;                  // all rows are of one query: they see the same tokens of every tile
    // The value scales so far, in tiles of which all rows see the same tokens: the exponents of the largest and of the smallest
    // that is not zero. A plain tile's smallest (as its f16 bits) lies above `unless`, or usual() looks at it.
    int e_most, e_least;
    uint32_t unless;
    // What only usual() and other than plain tiles need, in a word of each lane in shared memory:
    // kZeros: bit k: some token's scale of block k was zero, bit 8 + k: some token's was not (left at 0 as long as none was
    //   zero), as above in tiles of which all rows see the same tokens;
    // kOwn + r: for a row's other tiles the smallest exponent + 64, and from bit 8 on the same bits;
    // kLeast: the smallest exponent in any of these, kNone where a row is apart for good.
    enum : int { kZeros, kLeast, kOwn, kNotes = kOwn + LR };

    static constexpr uint32_t kQuad = KT ? 256 : 512, kOperands = MT * DB * 2 * kQuad;
    static constexpr uint32_t kQueries = kOperands + kNotes * 128;  // bytes of a warp's operands and notes

    __device__ __forceinline__ void init(uint32_t at) {
        lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
        queries = at + (uint32_t)lane * (kQuad / 32);
        asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
    }

    __device__ __forceinline__ void start(const Params& p, int b, int h, int row0, const Span& s) {
        const KvAttnArgs& a = p.a;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + n * 8 + g;
            const bool there = r < p.R;
            const int m = r / p.group;
            float x[DB][8];
            float big = 0.f;
            bool finite = true;
            const long long at_q = ((long long)b * a.M + m) * a.q_stride + (long long)(h * p.group + r - m * p.group) * D + 4 * t4;
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                float u[4] = {}, v[4] = {};
                if (there) {
                    load_q4(a.q, at_q + 32 * k, a.dtype, u);
                    load_q4(a.q, at_q + 32 * k + 16, a.dtype, v);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[k][j] = u[j], x[k][4 + j] = v[j];
                    finite = finite && fabsf(u[j]) < INFINITY && fabsf(v[j]) < INFINITY;
                    big = fmaxf(big, fmaxf(fabsf(u[j]), fabsf(v[j])));
                }
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const bool fine = (__ballot_sync(0xffffffffu, finite) >> (lane & ~3) & 15u) == 15u;
            // largest in [2^e, 2^(e+1)): scale by 2^(13 - e), as two factors that stay in range
            const int e = max((int)(__float_as_uint(big) >> 23), 1) - 127;
            const int k2 = big > 0.f && fine ? 13 - e : 0;
            const float f1 = pow2i(k2 / 2), f2 = pow2i(k2 - k2 / 2);
            factor[n] = fine ? (a.scale * 1.4426950408889634f) * pow2i(-(k2 / 2)) * pow2i(-(k2 - k2 / 2)) : qnan();
            seen_end[n] = s.n - a.M + min(m, a.M - 1) + 1;
            seen_lo[n] = a.window > 0 ? seen_end[n] - a.window : 0;
            const int mt = SPLIT ? n : n / 2, hi = SPLIT ? 0 : n % 2;
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                float xh[8], xl[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float y = fine ? (x[k][j] * f1) * f2 : 0.f;
                    if (j >= 4) y *= 0.0625f;
                    xh[j] = __half2float(__float2half_rn(y));
                    xl[j] = y - xh[j];
                }
                // words 0 and 2: row g, words 1 and 3: row g + 8 (the low parts of fp32 queries; the next group's rows of
                // 16-bit ones); KT: the column operand's two words
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t at = queries + (uint32_t)((mt * DB + k) * 2 + i) * kQuad;
                    const uint32_t a0 = pack_half2(xh[i], xh[i + 2]), a2 = pack_half2(xh[4 + i], xh[6 + i]);
                    if constexpr (SPLIT) {
                        sts_quad(at, a0, pack_half2(xl[i], xl[i + 2]), a2, pack_half2(xl[4 + i], xl[6 + i]));
                    } else if constexpr (KT) {
                        sts_word(at, a0);
                        sts_word(at + 4u, a2);
                    } else {
                        sts_word(at + 4u * hi, a0);
                        sts_word(at + 8u + 4u * hi, a2);
                    }
                }
            }
        }
        if constexpr (KT) {  // from row g to rows 2 t4, 2 t4 + 1
            const float f = factor[0];
            const int e = seen_end[0], lo = seen_lo[0];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int from = 8 * t4 + 4 * i;
                factor[i] = __shfl_sync(0xffffffffu, f, from);
                seen_end[i] = __shfl_sync(0xffffffffu, e, from), seen_lo[i] = __shfl_sync(0xffffffffu, lo, from);
            }
        }
        all_end = s.n - a.M + row0 / p.group + 1;
        all_lo = a.window > 0 ? max(s.lo, s.n - a.M + (min(p.R, row0 + ROWS) - 1) / p.group + 1 - a.window) : 0;
#pragma unroll
        for (int i = 0; i < NT * DB * 8; ++i) (&o[0][0][0][0])[i] = 0.f;
#pragma unroll
        for (int r = 0; r < LR; ++r) top[r] = -FLT_MAX, l[r] = 0.f, note(kOwn + r, kNoneSeen);
        note(kZeros, 0u), note(kLeast, 16u);
        e_most = -14, e_least = 16, unless = 0u;
        same = row0 / p.group == (min(p.R, row0 + ROWS) - 1) / p.group;
    }

    // The tile of tokens tok0 .. tok0 + 31 in the stage at shared address st.
    __device__ __forceinline__ void take(uint32_t st, int tok0) {
        const bool whole = tok0 >= all_lo && tok0 + kTile <= all_end;  // every row sees every token
        if (!whole || !tile<true>(st, tok0, true)) tile<false>(st, tok0, whole || same);
    }

    __device__ __forceinline__ uint32_t note_at(int i) const {
        return queries - (uint32_t)lane * (kQuad / 32 - 4) + kOperands + 128u * (uint32_t)i;
    }
    __device__ __forceinline__ uint32_t note(int i) const {
        uint32_t w[1];
        lds_own<1>(note_at(i), w);
        return w[0];
    }
    __device__ __forceinline__ void note(int i, uint32_t w) const { sts_word(note_at(i), w); }

    // Whether a whole tile is plain although it has zeros among its value scales (of this lane's token: own), or there were
    // zeros or tiles that not all rows saw alike before it: the zeros must be whole blocks that were always zero. Notes them,
    // and leaves in lo the smallest exponent (as bits) of the other scales.
    __device__ __forceinline__ bool usual(const uint32_t (&own)[DB / 2], uint32_t hi, uint32_t& lo) {
        uint32_t zeros = note(kZeros);
        if (lo == 0u || (zeros & 255u) != 0u) {
            uint32_t blocks = 0u, least = 0x7C00u;
            bool fits = true;
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                const uint32_t x = own[k / 2] >> (16 * (k % 2)) & 0x7FFFu;
                blocks |= x == 0u ? 1u << k : 256u << k;
                fits = fits && (x == 0u || x >= 0x0400u);
                least = x == 0u ? least : min(least, x & 0x7C00u);
            }
#pragma unroll
            for (int r = 0; r < LR; ++r) fits = fits && note(kOwn + r) == kNoneSeen;
            zeros = __reduce_or_sync(0xffffffffu, blocks) | (zeros == 0u && e_least < 16 ? 0xFF00u : zeros);
            if (!__all_sync(0xffffffffu, fits) || (zeros & zeros >> 8 & 255u) != 0u) return false;
            lo = __reduce_min_sync(0xffffffffu, least);
        }
        const int e_before = min(e_least, (int)note(kLeast));
        if (max(e_most, (int)(hi >> 10) - 15) - min(e_before, (int)(lo >> 10) - 15) > kRange) return false;
        note(kZeros, zeros);
        unless = 0xFFFFu;
        return true;
    }

    // PLAIN: a tile that every row sees whole, of finite normal value scales, without a row that is apart; false, with nothing
    // changed, where it is not. Else any tile; alike: all rows see the same of its tokens.
    template <bool PLAIN>
    __device__ __forceinline__ bool tile(uint32_t st, int tok0, bool alike) {
        constexpr bool MASKED = !PLAIN;
        const int own_row = row_of_lane<KT>(lane);
        const uint32_t codes = st + (uint32_t)(own_row * G::kRow + swizzle<DB>(own_row) * 16);  // chunk k: codes ^ (16 k)
        uint32_t own[2][DB / 2];  // the scales of this lane's token
        const uint32_t own_at = st + (uint32_t)(2 * G::kCodes + lane * DB * 2);
        lds_own<DB / 2>(own_at, own[0]);
        lds_own<DB / 2>(own_at + G::kScales, own[1]);
        uint32_t kw[DB][4];
#pragma unroll
        for (int k = 0; k < DB; ++k) ldsm4(codes ^ (uint32_t)(16 * k), kw[k]);
        const float offset_was = (float)(e_most - 14);
        bool apart[LR], some_apart = false;
        if constexpr (PLAIN) {
            uint32_t most = own[1][0] & 0x7C007C00u, least = most;
#pragma unroll
            for (int k = 1; k < DB / 2; ++k) {
                const uint32_t e = own[1][k] & 0x7C007C00u;
                most = half_max(most, e), least = half_min(least, e);
            }
            const uint32_t hi = __reduce_max_sync(0xffffffffu, max(most & 0xFFFFu, most >> 16));
            uint32_t lo = __reduce_min_sync(0xffffffffu, min(least & 0xFFFFu, least >> 16));
            if (hi >= 0x7C00u || (lo <= unless && !usual(own[1], hi, lo))) return false;
            const int e_hi = max(e_most, (int)(hi >> 10) - 15), e_lo = min(e_least, (int)(lo >> 10) - 15);
            if (e_hi - e_lo > kRange) return false;
            e_most = e_hi, e_least = e_lo;
        }
        if constexpr (MASKED) {
            int hi = -100, lo = 16;  // of this lane's token
            uint32_t blocks = 0u;
#pragma unroll
            for (int k = 0; k < DB; ++k) {
                const float2 d = to_float2(own[1][k / 2]);
                const float x = fabsf(k % 2 ? d.y : d.x);
                blocks |= x == 0.f ? 1u << k : 256u << k;
                const int e = (int)(__float_as_uint(x) >> 23) - 127;
                if (x > 0.f && x < INFINITY) hi = max(hi, e), lo = min(lo, e);
            }
            uint32_t zeros = note(kZeros), e_own[LR];
#pragma unroll
            for (int r = 0; r < LR; ++r) e_own[r] = note(kOwn + r);
            if (zeros == 0u && e_least < 16) zeros = 0xFF00u;  // so far no zeros
            if (alike) {
                const bool seen = tok0 + lane >= seen_lo[0] && tok0 + lane < seen_end[0];
                e_most = max(e_most, __reduce_max_sync(0xffffffffu, seen ? hi : -100));
                e_least = min(e_least, __reduce_min_sync(0xffffffffu, seen ? lo : 16));
                zeros |= __reduce_or_sync(0xffffffffu, seen ? blocks : 0u);
            } else {  // a token's word in the place of its values' scales
                sts_word(own_at + G::kScales, (uint32_t)(lo + 64) | blocks << 8);
                __syncwarp();
                const auto joined = [](uint32_t a, uint32_t b) { return min(a & 255u, b & 255u) | ((a | b) & ~255u); };
#pragma unroll
                for (int j = 0; j < (KT ? 4 : 8); ++j) {
                    const int in = (KT ? 4 * g : 8 * t4) + j;
                    uint32_t word[1];
                    lds_own<1>(st + (uint32_t)(2 * G::kCodes + G::kScales + in * DB * 2), word);
#pragma unroll
                    for (int r = 0; r < LR; ++r)
                        if (tok0 + in >= seen_lo[r] && tok0 + in < seen_end[r]) e_own[r] = joined(e_own[r], word[0]);
                }
#pragma unroll
                for (int r = 0; r < LR; ++r)
#pragma unroll
                    for (int x = KT ? 4 : 1; x <= (KT ? 16 : 2); x <<= 1) e_own[r] = joined(e_own[r], __shfl_xor_sync(0xffffffffu, e_own[r], x));
            }
            note(kZeros, zeros);
            int least = 16;
#pragma unroll
            for (int r = 0; r < LR; ++r) {
                note(kOwn + r, e_own[r]);
                const uint32_t z = zeros | e_own[r] >> 8;
                const int e = min(e_least, (int)(e_own[r] & 255u) - 64);
                apart[r] = !alike || (z & z >> 8 & 255u) != 0u || e_most - e > kRange;
                some_apart = some_apart || apart[r];
                least = min(least, (z & z >> 8 & 255u) != 0u || (e_own[r] >> 8 & 255u) != 0u ? kNone : e);
            }
            least = __reduce_min_sync(0xffffffffu, least);
            note(kLeast, (uint32_t)least);
            if (!alike || (zeros & 255u) != 0u || e_most - least > kRange) unless = 0xFFFFu;
        }
        // This lane's token's scales become fp32 [K, V][block][token] in the place of the keys' codes, which are in
        // registers now: a lane then reads those of its eight tokens as they are used (converting them where they are used
        // would take 64 conversions, eight lanes the same ones).
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int k = 0; k < DB / 2; ++k) {
                const float2 d = to_float2(own[v][k]);
                const uint32_t to = st + (uint32_t)(((v * DB + 2 * k) * 32 + lane) * 4);
                sts_word(to, __float_as_uint(d.x));
                sts_word(to + 128u, __float_as_uint(d.y));
            }
        __syncwarp();
        // of block k: + 128 k, of the values' blocks + 128 (DB + k)
        const uint32_t scales = st + (uint32_t)(KT ? 16 * g : 32 * t4);
        // scores, in pairs that an instruction leaves side by side: sc[n][j] and sc[n][j + 1], j even, are of row g of group n
        // the tokens 8 t4 + j and 8 t4 + j + 1; KT: of rows 2 t4 and 2 t4 + 1 the token 4 g + j / 2
        float sc[NT][8];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) sc[n][j] = 0.f;
#pragma unroll
        for (int k = 0; k < DB; ++k) {
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t x[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) codes_of(kw[k][j], k1024, x[j]);
            if constexpr (KT) {
                uint32_t q[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) lds_words<2>(queries + (uint32_t)(k * 2 + i) * kQuad, q[i]);
                float c[2][4], kd[4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t rows[4] = {x[2 * m][2 * i], x[2 * m + 1][2 * i], x[2 * m][2 * i + 1], x[2 * m + 1][2 * i + 1]};
                        if (i == 0) mma(c[m], rows, q[i][0], q[i][1], zero);
                        else mma(c[m], rows, q[i][0], q[i][1], c[m]);
                    }
                lds_floats4(scales + (uint32_t)(128 * k), kd);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 y = ffma2(make_float2(c[j / 2][2 * (j % 2)], c[j / 2][2 * (j % 2) + 1]), make_float2(kd[j], kd[j]),
                                           make_float2(sc[0][2 * j], sc[0][2 * j + 1]));
                    sc[0][2 * j] = y.x, sc[0][2 * j + 1] = y.y;
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float c[4][4], kd[8];
                    uint32_t q[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) lds_words<4>(queries + (uint32_t)((mt * DB + k) * 2 + i) * kQuad, q[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma(c[j], q[0], x[j][0], x[j][1], zero);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma(c[j], q[1], x[j][2], x[j][3], c[j]);
                    lds_floats(scales + (uint32_t)(128 * k), kd);
                    __syncwarp();  // keeps the blocks' instructions apart, and with them the registers in use
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 d = make_float2(kd[2 * j], kd[2 * j + 1]);
                        if constexpr (SPLIT) {
                            const float2 both = fadd2(make_float2(c[j][0], c[j][1]), make_float2(c[j][2], c[j][3]));
                            const float2 y = ffma2(both, d, make_float2(sc[mt][2 * j], sc[mt][2 * j + 1]));
                            sc[mt][2 * j] = y.x, sc[mt][2 * j + 1] = y.y;
                        } else {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int n = 2 * mt + u;
                                const float2 y = ffma2(make_float2(c[j][2 * u], c[j][2 * u + 1]), d,
                                                       make_float2(sc[n][2 * j], sc[n][2 * j + 1]));
                                sc[n][2 * j] = y.x, sc[n][2 * j + 1] = y.y;
                            }
                        }
                    }
                }
            }
        }

        // row r of a lane (r < LR) has the scores sc[KT ? 0 : r][KT ? 2 j + r : j], j < PER
        constexpr int PER = KT ? 4 : 8;
        auto score = [&](int r, int j) -> float& { return sc[KT ? 0 : r][KT ? 2 * j + r : j]; };
        uint32_t seen[LR];  // bit j
#pragma unroll
        for (int r = 0; r < LR; ++r) seen[r] = 0u;
        if constexpr (MASKED) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int in = (KT ? 4 * g : 8 * t4) + j, t = tok0 + in;
#pragma unroll
                for (int r = 0; r < LR; ++r) {
                    if (t >= seen_lo[r] && t < seen_end[r]) seen[r] |= 1u << j;
                    else score(r, j) = -INFINITY;
                }
            }
        }
        const float offset = (float)(e_most - 14);
        float keep[LR], ref[LR];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < LR; ++r) {
            float m = score(r, 0);
#pragma unroll
            for (int j = 1; j < PER; ++j) m = fmaxf(m, score(r, j));
#pragma unroll
            for (int x = KT ? 4 : 1; x <= (KT ? 16 : 2); x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            const float was = top[r] + offset_was;
            top[r] = fmaxf(top[r], m * factor[r]);
            ref[r] = top[r] + offset;
            keep[r] = was - ref[r];
            moved = moved || was != ref[r];
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int r = 0; r < LR; ++r) keep[r] = ex2(keep[r]), l[r] *= keep[r];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float ka, kb;
                if constexpr (KT) {
                    ka = keep[0], kb = keep[1];
                } else {
                    ka = __shfl_sync(0xffffffffu, keep[n], 8 * t4);
                    kb = __shfl_sync(0xffffffffu, keep[n], 8 * t4 + 4);
                }
#pragma unroll
                for (int k = 0; k < DB; ++k) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) o[n][k][j][0] *= ka, o[n][k][j][1] *= kb, o[n][k][j][2] *= ka, o[n][k][j][3] *= kb;
                }
            }
        }
        weights<MASKED>(sc, seen, ref);
        if (MASKED && __any_sync(0xffffffffu, some_apart)) values<MASKED, MASKED>(codes, scales, sc, seen, apart);
        else values<MASKED, false>(codes, scales, sc, seen, apart);
        return true;
    }

    // Weights in the place of the scores; a token that is not seen weighs nothing (also where the query is not finite).
    template <bool MASKED>
    __device__ __forceinline__ void weights(float (&sc)[NT][8], const uint32_t (&seen)[LR], const float (&ref)[LR]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r0 = KT ? 0 : n, r1 = KT ? 1 : n;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float2 y = ffma2(make_float2(sc[n][j], sc[n][j + 1]), make_float2(factor[r0], factor[r1]), make_float2(-ref[r0], -ref[r1]));
                y.x = ex2(y.x), y.y = ex2(y.y);
                if (MASKED && !(seen[r0] >> (KT ? j / 2 : j) & 1u)) y.x = 0.f;
                if (MASKED && !(seen[r1] >> (KT ? j / 2 : j + 1) & 1u)) y.y = 0.f;
                sc[n][j] = y.x, sc[n][j + 1] = y.y;
                sum = fadd2(sum, y);
            }
            if constexpr (KT) l[0] += sum.x, l[1] += sum.y;
            else l[n] += sum.x + sum.y;
        }
    }

    // The weights sc of a tile times its values, added to the outputs. APART: for a row that is apart the tile's largest term
    // in each block is brought to 2^14, and the products are summed from zero and brought back; other rows keep their bits.
    template <bool MASKED, bool APART>
    __device__ __forceinline__ void values(uint32_t codes, uint32_t scales, const float (&sc)[NT][8], const uint32_t (&seen)[LR],
                                           const bool (&apart)[LR]) {
#pragma unroll
        for (int k = 0; k < DB; ++k) {
            uint32_t w[4], x[4][4];
            ldsm4_trans((codes ^ (uint32_t)(16 * k)) + G::kCodes, w);
#pragma unroll
            for (int u = 0; u < 4; ++u) codes_of(w[u], k1024, x[u]);
            // weight times value scale, as the column operand: row g, two tokens of matrix j
            float vd[8];
            if constexpr (KT) {
                float v[4];
                lds_floats4(scales + (uint32_t)(128 * (DB + k)), v);
#pragma unroll
                for (int j = 0; j < 4; ++j) vd[2 * j] = vd[2 * j + 1] = v[j];
            } else {
                lds_floats(scales + (uint32_t)(128 * (DB + k)), vd);
            }
            auto term = [&](int n, int j) {
                const int r0 = KT ? 0 : n, r1 = KT ? 1 : n;
                float2 y = __fmul2_rn(make_float2(sc[n][2 * j], sc[n][2 * j + 1]), make_float2(vd[2 * j], vd[2 * j + 1]));
                if constexpr (MASKED) {  // a masked token's scale may be anything
                    if (!(seen[r0] >> (KT ? j : 2 * j) & 1u)) y.x = 0.f;
                    if (!(seen[r1] >> (KT ? j : 2 * j + 1) & 1u)) y.y = 0.f;
                }
                return y;
            };
            float up[LR], down[LR];  // APART: the row's powers of two; down 0: it is not apart
            if constexpr (APART) {
#pragma unroll
                for (int r = 0; r < LR; ++r) up[r] = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 y = term(n, j);
                        const int r0 = KT ? 0 : n, r1 = KT ? 1 : n;
                        up[r0] = fmaxf(up[r0], fabsf(y.x)), up[r1] = fmaxf(up[r1], fabsf(y.y));
                    }
#pragma unroll
                for (int r = 0; r < LR; ++r) {
#pragma unroll
                    for (int x = KT ? 4 : 1; x <= (KT ? 16 : 2); x <<= 1) up[r] = fmaxf(up[r], __shfl_xor_sync(0xffffffffu, up[r], x));
                    const int e = max((int)(__float_as_uint(up[r]) >> 23), 30) - 127;  // below 2^-97 nothing is left to keep
                    up[r] = apart[r] ? pow2i(14 - e) : 1.f;
                    down[r] = apart[r] ? pow2i(e - 14) : 0.f;
                }
            }
            uint32_t hi[NT][4], lo[SPLIT ? NT : 1][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float2 y = term(n, j);
                    if constexpr (APART) y = __fmul2_rn(y, make_float2(up[KT ? 0 : n], up[KT ? 1 : n]));
                    hi[n][j] = pack_half2(y.x, y.y);
                    if constexpr (KT) hi[n][j] = turned_over(hi[n][j]);
                    if constexpr (SPLIT) {
                        const float2 back = to_float2(hi[n][j]);
                        lo[n][j] = pack_half2(y.x - back.x, y.y - back.y);
                    }
                }
            }
            const uint32_t rows[2][2][4] = {{{x[0][0], x[0][1], x[1][0], x[1][1]}, {x[0][2], x[0][3], x[1][2], x[1][3]}},
                                            {{x[2][0], x[2][1], x[3][0], x[3][1]}, {x[2][2], x[2][3], x[3][2], x[3][3]}}};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                auto add = [&](float (&to)[2][4]) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        mma(to[0], rows[u][0], hi[n][2 * u], hi[n][2 * u + 1], to[0]);
                        mma(to[1], rows[u][1], hi[n][2 * u], hi[n][2 * u + 1], to[1]);
                        if constexpr (SPLIT) {
                            mma(to[0], rows[u][0], lo[n][2 * u], lo[n][2 * u + 1], to[0]);
                            mma(to[1], rows[u][1], lo[n][2 * u], lo[n][2 * u + 1], to[1]);
                        }
                    }
                };
                if constexpr (APART) {
                    float from[2];  // of rows 2 t4, 2 t4 + 1, which the outputs are of
#pragma unroll
                    for (int i = 0; i < 2; ++i) from[i] = KT ? down[KT ? i : 0] : __shfl_sync(0xffffffffu, down[KT ? 0 : n], 8 * t4 + 4 * i);
                    float sum[2][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) sum[j][c] = from[c % 2] == 0.f ? o[n][k][j][c] : 0.f;
                    add(sum);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            o[n][k][j][c] = from[c % 2] == 0.f ? sum[j][c] : fmaf(sum[j][c], from[c % 2], o[n][k][j][c]);
                } else {
                    add(o[n][k]);
                }
            }
        }
    }

    // Row g's sum over the whole warp, and its reference: -infinity where it saw nothing. NaN where a score was above fp32's
    // range (every weight under an infinite reference is 0), and whatever was seen if bad.
    __device__ __forceinline__ void finish(bool bad, float (&ref)[NT]) {
        float of[LR];
#pragma unroll
        for (int r = 0; r < LR; ++r) of[r] = top[r] + (float)(e_most - 14);
        if constexpr (KT) {  // from rows 2 t4, 2 t4 + 1 back to row g
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            const float l0 = __shfl_sync(0xffffffffu, l[0], g >> 1), l1 = __shfl_sync(0xffffffffu, l[1], g >> 1);
            const float r0 = __shfl_sync(0xffffffffu, of[0], g >> 1), r1 = __shfl_sync(0xffffffffu, of[1], g >> 1);
            l[0] = g & 1 ? l1 : l0, of[0] = g & 1 ? r1 : r0;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (!KT) {
                l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
                l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
            }
            ref[n] = l[n] == 0.f ? -INFINITY : of[n];
            if (bad || of[n] == INFINITY) l[n] = qnan(), ref[n] = 0.f;
        }
    }

    // Calls fn(n, row, element, pair) for the pairs of neighbouring elements that this lane holds: row 8 n + 2 t4 + i.
    template <typename F>
    __device__ __forceinline__ void each_pair(F fn) const {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < DB; ++k)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float f = half ? 0.0625f : 1.f;
                        fn(n, i, 32 * k + 16 * half + 2 * g, make_float2(o[n][k][0][2 * half + i] * f, o[n][k][1][2 * half + i] * f));
                    }
    }
};

// A warp's ring of stages, and its copies into it.
template <int DB, int STAGES, bool KT>
struct Ring {
    using G = Geo<DB>;
    uint32_t base, in, out;  // shared addresses: of the ring, of the stage to fill next, of the stage to use next
    const uint8_t *k_src, *v_src;
    int lane;

    __device__ __forceinline__ void init(uint32_t at, const kv4_cache& c) {
        lane = threadIdx.x & 31;
        base = in = out = at;
        k_src = c.k_qs + (lane % DB) * 16, v_src = c.v_qs + (lane % DB) * 16;
    }
    static __device__ __forceinline__ uint32_t after(uint32_t st, uint32_t base) {
        st += G::kStage;
        return st == base + STAGES * G::kStage ? base : st;
    }
    // The 32 tokens' rows of the cache (row: this lane's token's; negative: zeros): chunk lane % DB of every (32 / DB)-th
    // token, and the scales of token `lane`.
    __device__ __forceinline__ void copy(const kv4_cache& c, int row) {
        const uint32_t ds = in + (uint32_t)(2 * G::kCodes + lane * DB * 2);
        auto copies = [&](auto all) {  // all: every token of the tile is read
            constexpr bool ALL = decltype(all)::value;
#pragma unroll
            for (int j = 0; j < DB; ++j) {
                const int tok = j * (32 / DB) + lane / DB, at = place<KT>(tok);
                const int r = __shfl_sync(0xffffffffu, row, tok);
                const long long off = (long long)(ALL ? r : max(r, 0)) * G::kRow;
                const uint32_t dst = in + (uint32_t)(at * G::kRow + ((lane % DB) ^ swizzle<DB>(at)) * 16);
                const uint32_t bytes = ALL || r >= 0 ? 16u : 0u;
                copy_async<16>(dst, k_src + off, bytes);
                copy_async<16>(dst + G::kCodes, v_src + off, bytes);
            }
            const long long off = (long long)(ALL ? row : max(row, 0)) * DB;
            const uint32_t bytes = ALL || row >= 0 ? DB * 2 : 0;
            copy_async<DB * 2>(ds, c.k_d + off, bytes);
            copy_async<DB * 2>(ds + G::kScales, c.v_d + off, bytes);
        };
        if (__all_sync(0xffffffffu, row >= 0)) copies(std::true_type());
        else copies(std::false_type());
    }
    __device__ __forceinline__ void filled() {
        cp_async_commit();
        in = after(in, base);
    }
    __device__ __forceinline__ void wait() {  // for the oldest stage
        cp_async_wait<STAGES - 2>();
        __syncwarp();
    }
    __device__ __forceinline__ void used() { out = after(out, base); }
};

enum : int { kSkip = -1, kBadPage = -2 };

// A token to copy: its page as the page table has it. It is looked up a tile ahead, and nothing is made of the loaded page
// before the next tile's copies (row()), so that nobody waits for the load.
struct Lookup {
    int page, h, t;  // t < 0: none is read

    __device__ __forceinline__ void token(const Params& p, const int* table, int head, int tok, int lo, int end) {
        const bool read = tok >= lo && tok < end;
        h = head;
        t = read ? tok : -1;
        page = 0;
        if (read) page = table[tok >> p.lp];
    }
    __device__ __forceinline__ void none() { page = h = 0, t = -1; }
    // The token's cache row, kSkip where none is read, kBadPage where its page is none.
    __device__ __forceinline__ int row(const Params& p) const {
        if (t < 0) return kSkip;
        if ((unsigned)page >= (unsigned)p.a.c.num_pages) return kBadPage;
        return ((page * p.a.c.num_kv_heads + h) << p.lp) + (t & (p.a.c.page_size - 1));  // below 2^31
    }
};

// ------------------------------------------------------------------------------------------------
// Whole items
// ------------------------------------------------------------------------------------------------

template <int DB, int NT, bool SPLIT, int COUNT>
__global__ void __launch_bounds__(ItemPlan<DB, NT, SPLIT, COUNT>::kWarps * 32, ItemPlan<DB, NT, SPLIT, COUNT>::kCtas)
kv4_attention_items_kernel(const Params p) {
    using G = Geo<DB>;
    using L = ItemPlan<DB, NT, SPLIT, COUNT>;
    constexpr int D = G::D, ROWS = 8 * NT, kItemWarps = L::kWarps;
    extern __shared__ __align__(128) unsigned char ring_memory[];
    __shared__ float join_ref[kItemWarps][ROWS], join_l[kItemWarps][ROWS];
    const KvAttnArgs& a = p.a;
    const int warp = threadIdx.x >> 5;
    Rows<DB, NT, SPLIT> w;
    Ring<DB, L::kStages, Rows<DB, NT, SPLIT>::KT> ring;
    constexpr uint32_t kWarpBytes = L::kStages * G::kStage + Rows<DB, NT, SPLIT>::kQueries;
    const uint32_t mine_at = smem_addr(ring_memory) + (uint32_t)warp * kWarpBytes;
    ring.init(mine_at, a.c);
    w.init(mine_at + L::kStages * G::kStage);
    grid_dependency_wait();
    grid_launch_dependents();

    const int item = blockIdx.x / p.splits, split = blockIdx.x - item * p.splits;
    const int h = item / p.chunks, b = blockIdx.y, row0 = (item - h * p.chunks) * ROWS;
    const Span s = span_of(a, a.seq_lens[b]);
    const int* table = a.block_table + (long long)b * a.max_pages;
    bool bad = s.bad;
    // this CTA's tiles of the item, and where they end
    const int tile0 = (int)((long long)s.tiles * split / p.splits), tile1 = (int)((long long)s.tiles * (split + 1) / p.splits);
    const int mine = max(tile1 - tile0 - warp + kItemWarps - 1, 0) / kItemWarps;
    const int first = s.first + tile0 * kTile, end = min(s.n, s.first + tile1 * kTile);
    int ahead = first + warp * kTile + w.lane;  // this lane's token of the next tile to look up
    auto lookup = [&] {
        Lookup x;
        x.token(p, table, h, ahead, s.lo, end);
        ahead += kItemWarps * kTile;
        return x;
    };
    auto copy = [&](const Lookup& x) {
        const int row = x.row(p);
        bad = bad || row == kBadPage;
        ring.copy(a.c, row);
    };
    Lookup ups[L::kStages];
#pragma unroll
    for (int i = 0; i < L::kStages; ++i) ups[i] = lookup();
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) {
        if (i < mine) copy(ups[i]);
        ring.filled();
    }
    Lookup next = ups[L::kStages - 1];
    w.start(p, b, h, row0, s);
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        ring.wait();
        if (i + L::kStages - 1 < mine) copy(next);
        ring.filled();
        next = lookup();
        w.take(ring.out, first + (i * kItemWarps + warp) * kTile);
        ring.used();
    }
    cp_async_wait<0>();
    bad = __any_sync(0xffffffffu, bad) != 0;
    float ref[NT];
    w.finish(bad, ref);
    if (bad && w.lane == 0) atomicOr(a.fault, s.bad ? (unsigned)kFaultBadLength : (unsigned)kFaultBadPage);
    __syncthreads();  // every warp's stages are free: the join uses their memory
    float* jo = reinterpret_cast<float*>(ring_memory);
    if (w.t4 == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) join_l[warp][8 * n + w.g] = w.l[n], join_ref[warp][8 * n + w.g] = ref[n];
    }
    w.each_pair([&](int n, int i, int e, float2 v) {
        *reinterpret_cast<float2*>(jo + (warp * ROWS + 8 * n + 2 * w.t4 + i) * G::kJoinRow + e) = v;
    });
    __syncthreads();
    float* part = p.part + ((long long)b * gridDim.x + blockIdx.x) * (ROWS * (D + 2));
    for (int idx = threadIdx.x; idx < ROWS * (D / 4); idx += kItemWarps * 32) {
        const int r = idx / (D / 4), d4 = idx % (D / 4);
        if (row0 + r >= p.R) continue;
        float rt = -INFINITY, lt = 0.f;
#pragma unroll
        for (int u = 0; u < kItemWarps; ++u) rt = fmaxf(rt, join_ref[u][r]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rt != -INFINITY) {
#pragma unroll
            for (int u = 0; u < kItemWarps; ++u) {
                if (join_ref[u][r] == -INFINITY) continue;  // saw nothing
                const float f = ex2(join_ref[u][r] - rt);
                const float4 x = *reinterpret_cast<const float4*>(jo + (u * ROWS + r) * G::kJoinRow + 4 * d4);
                lt = fmaf(join_l[u][r], f, lt);
                v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
            }
        }
        if (p.splits == 1) {
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
            store_out4(a, out_at(p, b, h, row0 + r, D) + 4 * d4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            if (a.lse && d4 == 0) a.lse[lse_at(p, b, h, row0 + r)] = lse_of(rt, lt);
        } else {
            *reinterpret_cast<float4*>(part + r * D + 4 * d4) = v;
            if (d4 == 0) part[ROWS * D + r] = rt, part[ROWS * D + ROWS + r] = lt;
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Streams
// ------------------------------------------------------------------------------------------------

// prefix[b] = cost (of one key head and chunk) of the sequences before b, prefix[B] = of all. An item costs its tiles and
// kItemCost for its start: where tiles alone were divided, the warps with many short sequences came last by far.
template <int THREADS>
__device__ __forceinline__ void scan_cost(const KvAttnArgs& a, long long* prefix) {
    __shared__ long long warp_sum[THREADS / 32];
    const int per = (a.B + THREADS - 1) / THREADS;
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

// The part of an item that lies in a warp's piece of the line: `count` tiles from tile0 on. A warp keeps its parts in
// shared memory (all lanes write the same values), because they are looked at only where an item begins or ends.
struct Part {
    long long item_at;  // where the item begins on the line: its start's cost, then its tiles
    int b, item;        // sequence, head * chunks + chunk
    int tile0, count;
    Span s;
};

__device__ __forceinline__ void cut(Part& part, const KvAttnArgs& a, int b, int item, long long item_at, long long begin, long long end) {
    const Span s = span_of(a, a.seq_lens[b]);
    part.b = b, part.item = item, part.item_at = item_at, part.s = s;
    part.tile0 = (int)max(begin - item_at - kItemCost, 0LL);
    part.count = (int)min(end - item_at - kItemCost, (long long)s.tiles) - part.tile0;
}
// The first part of the piece [begin, end); count <= 0: none (the piece ends in an item's start).
__device__ __forceinline__ void first_part(Part& part, const KvAttnArgs& a, const long long* prefix, int items, long long begin, long long end) {
    int b = 0;
    for (int step = kMaxB / 2; step > 0; step >>= 1)
        if (b + step < a.B && prefix[b + step] * items <= begin) b += step;
    const int cost = (int)(prefix[b + 1] - prefix[b]);
    const long long rem = begin - prefix[b] * items;
    const int item = (int)(rem / cost);
    cut(part, a, b, item, begin - (rem - (long long)item * cost), begin, end);
}
__device__ __forceinline__ void next_part(Part& part, const KvAttnArgs& a, int items, long long end) {
    const long long at = part.item_at + part.s.tiles + kItemCost;
    int b = part.b, item = part.item + 1;
    if (item == items) item = 0, ++b;
    __syncwarp();  // every lane has read the part
    if (at >= end) part.count = 0;
    else cut(part, a, b, item, at, at, end);
    __syncwarp();
}

template <int DB, int NT, bool SPLIT>
__global__ void __launch_bounds__(Plan<DB, NT, SPLIT>::kWarps * 32, 1) kv4_attention_streams_kernel(const Params p) {
    using G = Geo<DB>;
    using L = Plan<DB, NT, SPLIT>;
    constexpr int D = G::D, ROWS = 8 * NT;
    extern __shared__ __align__(128) unsigned char ring_memory[];
    __shared__ long long prefix[kMaxB + 1];
    __shared__ Part parts[L::kWarps][2];
    __shared__ long long ends[L::kWarps];
    const KvAttnArgs& a = p.a;
    const int warp = threadIdx.x >> 5;
    // warps of one SM take pieces that are far apart: an SM that gets a stretch of short items gets others too
    const int stream = warp * (int)gridDim.x + (int)blockIdx.x;
    Rows<DB, NT, SPLIT> w;
    Ring<DB, L::kStages, Rows<DB, NT, SPLIT>::KT> ring;
    constexpr uint32_t kWarpBytes = L::kStages * G::kStage + Rows<DB, NT, SPLIT>::kQueries;
    const uint32_t mine_at = smem_addr(ring_memory) + (uint32_t)warp * kWarpBytes;
    ring.init(mine_at, a.c);
    w.init(mine_at + L::kStages * G::kStage);
    grid_dependency_wait();
    grid_launch_dependents();
    scan_cost<L::kWarps * 32>(a, prefix);

    const int items = a.c.num_kv_heads * p.chunks;
    const long long total = prefix[a.B] * items;
    // an even share of the cost, no less than an item of one tile
    const long long share = max((total + p.warps - 1) / (long long)p.warps, (long long)(1 + kItemCost));
    Part &use = parts[warp][0], &fill = parts[warp][1];  // of the tile to use next, and of the tile to look up next
    {
        const long long begin = min(total, share * stream), end = min(total, begin + share);
        if (begin >= end) return;
        first_part(use, a, prefix, items, begin, end);
        fill = use;
        ends[warp] = end;
        __syncwarp();
        if (use.count <= 0) return;
    }
    int left = fill.count, ahead = fill.s.first + fill.tile0 * kTile + w.lane, ahead_lo = fill.s.lo, ahead_end = fill.s.n;
    const int* table = a.block_table + (long long)fill.b * a.max_pages;
    int fill_h = fill.item / p.chunks;
    auto lookup = [&](bool& some) {  // this lane's token of the next tile of the piece; some: there is a tile
        Lookup x;
        x.none();
        some = left > 0;
        if (!some) return x;
        x.token(p, table, fill_h, ahead, ahead_lo, ahead_end);
        ahead += kTile;
        if (--left == 0) {
            next_part(fill, a, items, ends[warp]);
            left = max(fill.count, 0);
            if (left > 0) {
                ahead = fill.s.first + fill.tile0 * kTile + w.lane, ahead_lo = fill.s.lo, ahead_end = fill.s.n;
                table = a.block_table + (long long)fill.b * a.max_pages;
                fill_h = fill.item / p.chunks;
            }
        }
        return x;
    };
    uint32_t bad_stages = 0u;  // bit i: the tile copied i tiles before the newest met a bad page
    auto copy = [&](bool some, const Lookup& x) {
        const int row = x.row(p);
        if (some) ring.copy(a.c, row);
        bad_stages = bad_stages << 1 | (some && row == kBadPage ? 1u : 0u);
        ring.filled();
    };
    Lookup ups[L::kStages];
    bool some[L::kStages];
#pragma unroll
    for (int i = 0; i < L::kStages; ++i) ups[i] = lookup(some[i]);
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) copy(some[i], ups[i]);
    Lookup next = ups[L::kStages - 1];
    bool next_some = some[L::kStages - 1];

#pragma unroll 1
    for (;;) {
        bool bad = use.s.bad;
        {
            const int h = use.item / p.chunks;
            w.start(p, use.b, h, (use.item - h * p.chunks) * ROWS, use.s);
        }
        int tok0 = use.s.first + use.tile0 * kTile;
        const int last = tok0 + use.count * kTile;
#pragma unroll 1
        for (; tok0 != last; tok0 += kTile) {
            ring.wait();
            bad = bad || (bad_stages >> (L::kStages - 2) & 1u);
            copy(next_some, next);
            next = lookup(next_some);
            w.take(ring.out, tok0);
            ring.used();
        }
        const int b = use.b, h = use.item / p.chunks, row0 = (use.item - h * p.chunks) * ROWS;
        bad = __any_sync(0xffffffffu, bad) != 0;
        float ref[NT];
        w.finish(bad, ref);
        if (bad && w.lane == 0) atomicOr(a.fault, use.s.bad ? (unsigned)kFaultBadLength : (unsigned)kFaultBadPage);
        if (use.count == use.s.tiles) {  // the whole item: its outputs
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float inv = w.l[n] == 0.f ? 0.f : 1.f / w.l[n];
                const int r = row0 + 8 * n + w.g;
                if (a.lse && w.t4 == 0 && r < p.R) a.lse[lse_at(p, b, h, r)] = lse_of(ref[n], w.l[n]);
                w.l[n] = inv;
            }
            long long to[NT][2];
            float inv[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = row0 + 8 * n + 2 * w.t4 + i;
                    inv[n][i] = __shfl_sync(0xffffffffu, w.l[n], 8 * w.t4 + 4 * i);
                    to[n][i] = r < p.R ? out_at(p, b, h, r, D) : -1;
                }
            w.each_pair([&](int n, int i, int e, float2 v) {
                if (to[n][i] < 0) return;
                v.x *= inv[n][i], v.y *= inv[n][i];
                const long long at = to[n][i] + e;
                if (a.dtype == Q4_F32) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = v;
                else if (a.dtype == Q4_F16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) = pack2(v.x, v.y, __half());
                else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) = pack2(v.x, v.y, __nv_bfloat16());
            });
            if (w.lane == 0) p.desc[b * items + use.item] = make_int2(1, 0);
        } else {
            // a part of an item that began before goes to slot 0
            const int slot = use.item_at + kItemCost < share * stream ? 0 : 1;
            float* part = p.part + ((long long)stream * 2 + slot) * (ROWS * (D + 2));
            if (w.t4 == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    part[ROWS * D + 8 * n + w.g] = ref[n], part[ROWS * D + ROWS + 8 * n + w.g] = w.l[n];
            }
            w.each_pair([&](int n, int i, int e, float2 v) {
                const int r = 8 * n + 2 * w.t4 + i;
                if (row0 + r < p.R) *reinterpret_cast<float2*>(part + r * D + e) = v;
            });
            if (use.tile0 == 0 && w.lane == 0)  // the item begins here: its join starts from this warp
                p.desc[b * items + use.item] = make_int2((int)((use.item_at + use.s.tiles + kItemCost - 1) / share) - stream + 1, stream * 2 + slot);
        }
        next_part(use, a, items, ends[warp]);
        if (use.count <= 0) break;
    }
    cp_async_wait<0>();
}

// Joins the parts of an item that was divided: block x item x of the call, ROWS / gridDim.y of its rows. A block's threads stand over rows, parts and groups of four elements; every sum has a fixed order.
constexpr int kJoinThreads = 256;
template <int DB, int NT, int RPB>  // RPB: rows a block
__global__ void __launch_bounds__(kJoinThreads) kv4_attention_join_kernel(const Params p) {
    constexpr int D = DB * 32, ROWS = 8 * NT, D4 = D / 4;
    constexpr int RT = RPB * D4 <= kJoinThreads ? RPB : kJoinThreads / D4;  // rows at a time
    constexpr int PT = kJoinThreads / (RT * D4);                            // parts at a time
    __shared__ float4 so[PT][RT][D4];
    __shared__ float sl[PT][RT], sm[PT][RT];
    grid_dependency_wait();
    grid_launch_dependents();
    const int items = p.a.c.num_kv_heads * p.chunks, stride = ROWS * (D + 2);
    const int b = blockIdx.x / items, item = blockIdx.x - b * items;
    const int h = item / p.chunks, row0 = (item - h * p.chunks) * ROWS;
    int n = p.splits, slot = 0;
    const float* part0 = p.part + (long long)blockIdx.x * n * stride;  // split items: their parts follow each other
    if (p.warps) {  // streams: a slot of the first piece, then slot 0 of the next pieces
        const int2 ds = p.desc[blockIdx.x];
        n = ds.x, slot = ds.y & 1;
        if (n <= 1) return;
        part0 = p.part + (long long)ds.y * stride;
    }
    auto part = [&](int i) { return part0 + (long long)(p.warps ? (i == 0 ? 0 : 2 * i - slot) : i) * stride; };
    const int d4 = threadIdx.x % D4, rt = threadIdx.x / D4 % RT, pt = threadIdx.x / (D4 * RT);
    for (int r0 = blockIdx.y * RPB; r0 < (int)(blockIdx.y + 1) * RPB; r0 += RT) {
        const int r = r0 + rt;
        if (row0 + r0 >= p.R) break;  // the same for the whole block
        // a thread's share of the parts, eight in flight, each under the largest reference so far (a part that saw nothing
        // has reference -infinity and weighs 0)
        float top = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAhead = 8;
        for (int i0 = pt; i0 < n; i0 += PT * kAhead) {
            float4 o[kAhead];
            float ref[kAhead], pl[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * PT;
                ref[u] = -INFINITY, pl[u] = 0.f, o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n) {
                    const float* x = part(i);
                    o[u] = *reinterpret_cast<const float4*>(x + r * D + 4 * d4);
                    ref[u] = x[ROWS * D + r], pl[u] = x[ROWS * D + ROWS + r];
                }
            }
            float nt = top;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) nt = fmaxf(nt, ref[u]);
            if (nt != -INFINITY) {
                const float keep = ex2(top - nt);
                l *= keep, v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const float f = ex2(ref[u] - nt);
                    l = fmaf(pl[u], f, l);
                    v.x = fmaf(o[u].x, f, v.x), v.y = fmaf(o[u].y, f, v.y), v.z = fmaf(o[u].z, f, v.z), v.w = fmaf(o[u].w, f, v.w);
                }
                top = nt;
            }
        }
        if constexpr (PT > 1) {
            so[pt][rt][d4] = v;
            if (d4 == 0) sl[pt][rt] = l, sm[pt][rt] = top;
            __syncthreads();
            if (pt == 0) {
                float all = top;
#pragma unroll
                for (int u = 1; u < PT; ++u) all = fmaxf(all, sm[u][rt]);
                if (all != -INFINITY) {
                    const float keep = ex2(top - all);
                    l *= keep, v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
                    for (int u = 1; u < PT; ++u) {
                        const float4 o = so[u][rt][d4];
                        const float f = ex2(sm[u][rt] - all);
                        l = fmaf(sl[u][rt], f, l);
                        v.x = fmaf(o.x, f, v.x), v.y = fmaf(o.y, f, v.y), v.z = fmaf(o.z, f, v.z), v.w = fmaf(o.w, f, v.w);
                    }
                    top = all;
                }
            }
        }
        if (pt == 0 && row0 + r < p.R) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            store_out4(p.a, out_at(p, b, h, row0 + r, D) + 4 * d4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            if (p.a.lse && d4 == 0) p.a.lse[lse_at(p, b, h, row0 + r)] = lse_of(top, l);
        }
        __syncthreads();
    }
}

// Groups of 8 rows that a warp holds: two where there are more than 8 rows and the outputs fit the registers.
int row_groups(int M, int group, int D) { return M * group > 8 && D < 256 ? 2 : 1; }

// Items (whole, or split evenly over up to two CTAs an SM, one for every 256 tokens that the page table or the window admits)
// where the page table and the window let no sequence read more than kItemTokens, for a single sequence, and for few items of
// up to kSplitTokens; streams otherwise. The host knows what is admitted, not the lengths: a table much wider than its
// sequence costs CTAs without a tile, and the join (one sequence of 100 tokens, fp32, 4 key heads of 128: 5.7 us behind a table
// for 128 tokens, 6.9, 7.6 and 8.5 us behind one for 2,048, 16,384 and 131,072; of 16,384 tokens 9.8 and, for 131,072, 10.9).
// The streams' scan, their second launch and its join cost 5 to 8 us more than a launch of whole items, and do not mind the
// lengths, where the CTAs with the longest of ragged items are waited for. 8 key heads of 128, bf16, items and streams: 8
// sequences of 100 tokens 6.3 and 14.2 us, of 1500 tokens 11 and 16 us; 64 of 1000 tokens 25 and 29 us; 64 with a window of
// 512 tokens 16 and 22 us; one of 131001 tokens 38 and 46 us; 64 ragged ones up to 2000 tokens 33 and 30 us, up to 8192
// tokens 107 and 71 us.
constexpr long long kItemTokens = 1024;
constexpr long long kSplitTokens = 8192;

template <typename F>
auto with_plan(int D, int nt, bool split, F fn) {
    auto by_split = [&](auto db, auto n) {
        return split ? fn(db, n, std::true_type()) : fn(db, n, std::false_type());
    };
    using one = std::integral_constant<int, 1>;
    using two = std::integral_constant<int, 2>;
    using four = std::integral_constant<int, 4>;
    if (D == 64) return nt == 2 ? by_split(two(), two()) : by_split(two(), one());
    if (D == 128) return nt == 2 ? by_split(four(), two()) : by_split(four(), one());
    return by_split(std::integral_constant<int, 8>(), one());
}

// Launches a kernel with `ring` bytes of dynamic shared memory, which it is allowed once on each device.
template <auto kKernel>
cudaError_t launch_with_ring(dim3 grid, int threads, uint32_t ring, const DeviceInfo& di, cudaStream_t s, const Params& p) {
    static std::atomic<bool> allowed[64];
    if (!allowed[di.device & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
        if (e != cudaSuccess) return e;
        allowed[di.device & 63].store(true, std::memory_order_relaxed);
    }
    return launch_grid(kKernel, grid, dim3((unsigned)threads), ring, s, launch_overlap(), p);
}

}  // namespace

size_t kv4_attention_workspace_bytes(int M, int group, int heads, int D, int dtype, int sm_count) {
    const int nt = row_groups(M, group, D);
    return with_plan(D, nt, dtype == Q4_F32, [&](auto db, auto n, auto split) {
        constexpr int DB = decltype(db)::value, NT = decltype(n)::value;
        const size_t warps = (size_t)sm_count * Plan<DB, NT, decltype(split)::value>::kWarps;
        const size_t items = (size_t)heads * ((M * group + 8 * NT - 1) / (8 * NT));
        return warps * 2 * 8 * NT * (DB * 32 + 2) * sizeof(float) + kMaxB * items * sizeof(int2);
    });
}

cudaError_t launch_kv4_attention(const KvAttnArgs& a, void* workspace, const DeviceInfo& di, cudaStream_t s) {
    const int sm_count = di.sm_count;
    const int group = a.Hq / a.c.num_kv_heads, nt = row_groups(a.M, group, a.c.head_dim);
    return with_plan(a.c.head_dim, nt, a.dtype == Q4_F32, [&](auto db, auto n, auto split) {
        constexpr int DB = decltype(db)::value, NT = decltype(n)::value;
        constexpr bool SPLIT = decltype(split)::value;
        using G = Geo<DB>;
        using L = Plan<DB, NT, SPLIT>;
        Params p;
        p.a = a;
        p.warps = sm_count * L::kWarps;
        p.part = static_cast<float*>(workspace);
        p.desc = reinterpret_cast<int2*>(p.part + (size_t)p.warps * 2 * 8 * NT * (DB * 32 + 2));
        p.R = group * a.M;
        p.group = group;
        p.chunks = (p.R + 8 * NT - 1) / (8 * NT);
        p.splits = 1;
        p.lp = 0;
        while ((1 << p.lp) < a.c.page_size) ++p.lp;
        const int items = a.c.num_kv_heads * p.chunks;
        auto join = [&](unsigned blocks, bool few) {  // few items: a row a block
            // It may be scheduled while the parts are computed, whatever the overlap setting: both are this call's own.
            return few ? launch_grid(kv4_attention_join_kernel<DB, NT, 1>, dim3(blocks, 8 * NT), dim3(kJoinThreads), 0, s, true, p)
                       : launch_grid(kv4_attention_join_kernel<DB, NT, 8 * NT>, dim3(blocks), dim3(kJoinThreads), 0, s, true, p);
        };
        // the tokens that an item reads at most
        const long long held = (long long)a.max_pages * a.c.page_size, call_items = (long long)items * a.B;
        const long long most = a.window > 0 ? std::min(held, (long long)a.window + a.M - 1) : held;
        if (most <= kItemTokens || a.B == 1 || (most <= kSplitTokens && call_items <= sm_count)) {
            p.warps = 0;
            p.splits = (int)std::max(1LL, std::min(2LL * sm_count / call_items, most / (8 * kTile)));
            auto go = [&](auto count) {
                constexpr int COUNT = decltype(count)::value;
                using I = ItemPlan<DB, NT, SPLIT, COUNT>;
                constexpr int kRing = I::kWarps * (I::kStages * G::kStage + (int)Rows<DB, NT, SPLIT>::kQueries);
                static_assert(kRing >= I::kWarps * 8 * NT * G::kJoinRow * 4, "the join must fit in the rings");
                return launch_with_ring<kv4_attention_items_kernel<DB, NT, SPLIT, COUNT>>(
                    dim3((unsigned)(items * p.splits), (unsigned)a.B), I::kWarps * 32, kRing, di, s, p);
            };
            // more CTAs than two an SM run in kMany where 128 registers do; from eight an SM on, CTAs of two warps take over,
            // each warp with twice the tiles and half the starts: 256 sequences of 64 tokens 21 and 15 us, of 300 tokens 33 and
            // 28 us, but 64 sequences of 200 tokens 10.1 and 10.7 us (8 key heads of 128, bf16)
            constexpr bool kFour = DB == 2 || (DB == 4 && NT == 1);
            const long long ctas = call_items * p.splits;
            cudaError_t e;
            if (kFour && ctas >= 8LL * sm_count) e = go(std::integral_constant<int, kFour ? kCrowd : kFew>());
            else if (kFour && ctas > 2LL * sm_count) e = go(std::integral_constant<int, kFour ? kMany : kFew>());
            else e = go(std::integral_constant<int, kFew>());
            if (e == cudaSuccess && p.splits > 1) e = join((unsigned)call_items, true);
            return e;
        }
        cudaError_t e = launch_with_ring<kv4_attention_streams_kernel<DB, NT, SPLIT>>(
            dim3((unsigned)sm_count), L::kWarps * 32, L::kWarps * (L::kStages * G::kStage + (int)Rows<DB, NT, SPLIT>::kQueries), di, s, p);
        if (e == cudaSuccess) e = join((unsigned)call_items, call_items <= 64);
        return e;
    });
}

}  // namespace q4
