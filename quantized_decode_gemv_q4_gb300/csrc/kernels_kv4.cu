// Writing keys and values into the 4-bit cache, and reading them back.
//
// A cache row is a planar Q4 row (32-element blocks, byte j of a block holds element j in its low and j + 16 in its
// high nibble, value (code - 8) * d). A block is quantised as
//   d = f16(min(max|x| / 7, 65504)),  code = 8 + clamp(nearest(x / d), -7, 7)   (ties to even; d = 0: code 8),
// so |x - (code - 8) d| <= d / 2 plus the rounding of d itself. A block that holds a NaN or an infinity gets d = NaN
// (and codes 8): it reads back as NaN.
#include "kv_common.cuh"

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxThreads = 512;
// Tokens of a thread where there are many pieces (three for each resident thread of the device, so that fewer threads with
// more in flight still fill it): 16384 bf16 tokens of 8 heads of 128, write and read back, take 48 us with one token a
// thread, 37 us with four (26 us for the bytes; the write's 17 instructions an element bind); the read of 50001 tokens 65
// and 44 us (39 us for the bytes).
template <typename T>
constexpr int kTokens = 8 / (int)sizeof(T);
constexpr long long kManyPieces = 1LL << 20;

// A thread holds 16 elements of a 32-element block, those of 8 code bytes: elements 8 s .. 8 s + 7 (low nibbles) and
// 16 + 8 s .. (high nibbles) of side s = 0, 1; so a block's two threads write whole 32-byte sectors of values, and their
// only exchange is the block's maximum. A token's Hkv * D / 8 pieces run over its K heads, then its V heads. A thread
// takes the same piece of U tokens, all of whose loads are in flight at once.
struct Piece {
    bool v;
    int el;          // first low element in the token's row
    int head, blk, side;
};
__device__ __forceinline__ Piece piece_of(const kv4_cache& c, int u) {
    Piece q;
    const int half = c.num_kv_heads * c.head_dim / 16;  // pieces of K, and of V
    q.v = u >= half;
    const int in = q.v ? u - half : u, per_head = c.head_dim / 16;
    q.head = in / per_head;
    const int in_row = in - q.head * per_head;
    q.blk = in_row >> 1, q.side = in_row & 1;
    q.el = q.head * c.head_dim + 32 * q.blk + 8 * q.side;
    return q;
}

// nearest(x / d) for d an f16 value > 0, ties to even, exactly: r = rint(x * (1 / d)) is the nearest or next to it,
// and x - r d is exact in fp32 (r d has 15 bits, and the difference is below 2^24 units of the smaller operand's
// last place), so comparing it with d / 2 settles it. Where |x| > 7.5 d the result only has to be past 7.
__device__ __forceinline__ float nearest_quotient(float x, float d, float inv) {
    float r = rintf(fminf(fmaxf(x * inv, -8.f), 8.f));
    const float e = fmaf(-r, d, x), h = 0.5f * d;
    const bool odd = (__float2int_rn(r) & 1) != 0;
    if (e > h || (e == h && odd)) r += 1.f;
    if (e < -h || (e == -h && odd)) r -= 1.f;
    return fminf(fmaxf(r, -7.f), 7.f);
}

// The eight code bytes (8 + r_lo) + 16 (8 + r_hi) of a thread's elements with nearest_quotient, one after the other from
// memory: rarely needed, so kept small.
template <typename T>
__device__ __noinline__ uint2 exact_bytes(const T* src, float d) {
    unsigned long long w = 0ull;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
        const float a = nearest_quotient((float)src[j], d, 1.f / d), b = nearest_quotient((float)src[16 + j], d, 1.f / d);
        w |= (unsigned long long)(136 + __float2int_rn(a) + 16 * __float2int_rn(b)) << (8 * j);
    }
    return make_uint2((uint32_t)w, (uint32_t)(w >> 32));
}

// The same from low elements lo and high elements hi in registers. Adding 1.5 * 2^23 leaves a rounded quotient as a float
// (and, the second time, the byte in the low bits).
//   fp32: the quotient by an approximate reciprocal; exact_bytes is left to a thread that met a value within 2^-18 of a
//   border, which random values are once in 2^18.
//   16-bit types: a value of at most 11 bits lies on a border (k + 1/2) d of at most 15 bits, or 2^-16 away. One Newton
//   step gives the quotient to 2^-22, and exactly where it lies on a border, which is common (one block in 25: the scale
//   of a bf16 maximum divisible by 7 is exact).
// Either way exact_bytes takes the blocks whose scale leaves quotients past 7.5 (below f16's normal range, or capped).
template <typename T>
__device__ __forceinline__ uint2 code_bytes(const float (&lo)[8], const float (&hi)[8], float top, float d, const T* src) {
    constexpr float kMagic = 12582912.f;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
    float off = 0.f;
    uint32_t byte[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float a, b;
        if constexpr (sizeof(T) == 4) {
            a = fmaf(lo[j], inv, kMagic) - kMagic, b = fmaf(hi[j], inv, kMagic) - kMagic;
            off = fmaxf(off, fmaxf(fabsf(fmaf(-a, d, lo[j])), fabsf(fmaf(-b, d, hi[j]))));
        } else {
            const float x = lo[j] * inv, y = hi[j] * inv;
            a = (fmaf(fmaf(-x, d, lo[j]), inv, x) + kMagic) - kMagic;
            b = (fmaf(fmaf(-y, d, hi[j]), inv, y) + kMagic) - kMagic;
        }
        byte[j] = __float_as_uint(fmaf(b, 16.f, a) + (kMagic + 136.f));
    }
    if (off >= 0.5f * d * (1.f - 0x1p-18f) || d < 0x1p-14f || top > 7.f * 65504.f) return exact_bytes(src, d);
    uint2 w;
    w.x = __byte_perm(__byte_perm(byte[0], byte[1], 0x0040), __byte_perm(byte[2], byte[3], 0x0040), 0x5410);
    w.y = __byte_perm(__byte_perm(byte[4], byte[5], 0x0040), __byte_perm(byte[6], byte[7], 0x0040), 0x5410);
    return w;
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight elements from the 16-byte words that they were loaded in.
__device__ __forceinline__ void widen8(const uint4* w, float (&x)[8], float) {
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]);
}
template <typename T>
__device__ __forceinline__ void widen8(const uint4* w, float (&x)[8], T tag) {
    const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(v[i], tag);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}

template <typename T, int U>
__global__ void __launch_bounds__(kMaxThreads) kv4_write_kernel(const KvRowsArgs p) {
    const int pieces = p.c.num_kv_heads * p.c.head_dim / 8;
    const int t0 = ((int)blockIdx.x * (int)blockDim.y + (int)threadIdx.y) * U, slots = p.c.num_pages * p.c.page_size;
    grid_dependency_wait();
    grid_launch_dependents();
    int slot[U];
#pragma unroll
    for (int i = 0; i < U; ++i) slot[i] = t0 + i < p.T ? p.slots[t0 + i] : -1;
    for (int u0 = 0; u0 < pieces; u0 += (int)blockDim.x) {  // every thread of a warp takes part in the shuffles
        const int u = u0 + (int)threadIdx.x;
        const bool active = u < pieces;
        const Piece q = piece_of(p.c, active ? u : 0);
        const T* src = static_cast<const T*>(q.v ? p.v : p.k) + q.el;
        const long long stride = q.v ? p.v_stride : p.k_stride;
        constexpr int W = (int)sizeof(T) / 2;  // 16-byte words of 8 elements
        uint4 raw[U][2 * W];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool read = active && t0 + i < p.T;
            const uint4 *lo = reinterpret_cast<const uint4*>(src + (t0 + i) * stride), *hi = reinterpret_cast<const uint4*>(src + (t0 + i) * stride + 16);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                raw[i][j] = read ? lo[j] : make_uint4(0u, 0u, 0u, 0u);
                raw[i][W + j] = read ? hi[j] : make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float lo[8], hi[8];
            widen8(&raw[i][0], lo, T());
            widen8(&raw[i][W], hi, T());
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max_or_nan(top, max_or_nan(fabsf(lo[j]), fabsf(hi[j])));
            top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
            const bool finite = top < INFINITY;
            const __half dh = __float2half_rn(fminf(__fdiv_rn(top, 7.f), 65504.f));
            const float d = __half2float(dh);
            const uint2 w = finite && d > 0.f ? code_bytes(lo, hi, top, d, src + (t0 + i) * stride)
                                              : make_uint2(0x88888888u, 0x88888888u);
            if (active && slot[i] >= 0 && slot[i] < slots) {
                const int page = slot[i] >> p.lp, off = slot[i] & (p.c.page_size - 1);
                const long long row = cache_row(p.c, page, q.head, off);
                *reinterpret_cast<uint2*>((q.v ? p.c.v_qs : p.c.k_qs) + row * (p.c.head_dim / 2) + q.blk * 16 + q.side * 8) = w;
                if (q.side == 0)
                    (q.v ? p.c.v_d : p.c.k_d)[row * (p.c.head_dim / 32) + q.blk] = finite ? __half_as_ushort(dh) : (unsigned short)0x7E00u;
            }
        }
    }
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (slot[i] >= slots) atomicOr(p.fault, (unsigned)kFaultBadSlot);
    }
}

// The four low and four high elements of a word of codes. A code at bits p .. p + 3 (p <= 16) under the pattern of 2^23 is
// 2^23 + code * 2^p, so a difference leaves (code - 8) * 2^p exactly and a product with d * 2^-p, exact as well (15 bits),
// the value: no shift and no conversion from integers, which cost the reader more than its bytes did.
__device__ __forceinline__ void value_words(uint32_t w, float d, float* lo, float* hi) {
    const uint32_t s = w >> 12;
    auto value = [&](uint32_t v, int p) {
        const float x = __uint_as_float((v & (15u << p)) | 0x4B000000u) - (8388608.f + (float)(8 << p));
        return x * (d * __int_as_float((127 - p) << 23));
    };
    lo[0] = value(w, 0), lo[1] = value(w, 8), lo[2] = value(w, 16), lo[3] = value(s, 12);
    hi[0] = value(w, 4), hi[1] = value(w, 12), hi[2] = value(s, 8), hi[3] = value(s, 16);
}

template <typename T, int U>
__global__ void __launch_bounds__(kMaxThreads) kv4_read_kernel(const KvRowsArgs p) {
    const int pieces = p.c.num_kv_heads * p.c.head_dim / 8;
    const int t0 = ((int)blockIdx.x * (int)blockDim.y + (int)threadIdx.y) * U, slots = p.c.num_pages * p.c.page_size;
    grid_dependency_wait();
    grid_launch_dependents();
    int slot[U];
#pragma unroll
    for (int i = 0; i < U; ++i) slot[i] = t0 + i < p.T ? p.slots[t0 + i] : -1;
    for (int u = (int)threadIdx.x; u < pieces; u += (int)blockDim.x) {
        const Piece q = piece_of(p.c, u);
        T* dst = static_cast<T*>(q.v ? p.v : p.k);
        if (!dst) continue;
        dst += q.el;
        const long long stride = q.v ? p.v_stride : p.k_stride;
        uint2 w[U];
        float d[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool there = slot[i] >= 0 && slot[i] < slots;
            const int at = there ? slot[i] : 0, page = at >> p.lp, off = at & (p.c.page_size - 1);
            const long long row = cache_row(p.c, page, q.head, off);
            w[i] = *reinterpret_cast<const uint2*>((q.v ? p.c.v_qs : p.c.k_qs) + row * (p.c.head_dim / 2) + q.blk * 16 + q.side * 8);
            d[i] = f16_bits_to_f32((q.v ? p.c.v_d : p.c.k_d)[row * (p.c.head_dim / 32) + q.blk]);
            if (!there) d[i] = qnan();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (slot[i] < 0) continue;
            float lo[8], hi[8];
            value_words(w[i].x, d[i], &lo[0], &hi[0]);
            value_words(w[i].y, d[i], &lo[4], &hi[4]);
            store_floats(dst + (t0 + i) * stride, lo);
            store_floats(dst + (t0 + i) * stride + 16, hi);
        }
    }
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (slot[i] >= slots) atomicOr(p.fault, (unsigned)kFaultBadSlot);
    }
}

// A block's threads: x over a token's pieces (a multiple of 4), y over groups of U tokens so that short tokens share a
// block; a whole number of warps, at most kMaxThreads.
dim3 rows_block(int pieces) {
    if (pieces >= kThreads) return dim3(kThreads);
    if (pieces >= 64) {
        const int x = (pieces + 31) / 32 * 32;
        return dim3((unsigned)x, (unsigned)(kThreads / x));
    }
    int y = kThreads / pieces;
    if (pieces % 32) y = (y + 7) / 8 * 8;
    return dim3((unsigned)pieces, (unsigned)y);
}

template <int N, typename F1, typename F4>
cudaError_t launch_rows(const KvRowsArgs& a, cudaStream_t s, F1 one, F4 four) {
    const int pieces = a.c.num_kv_heads * a.c.head_dim / 8;
    const dim3 block = rows_block(pieces);
    const bool many = (long long)a.T * pieces >= kManyPieces;
    const int tokens = (int)block.y * (many ? N : 1);
    const dim3 grid((unsigned)((a.T + tokens - 1) / tokens));
    return many ? launch_grid(four, grid, block, 0, s, launch_overlap(), a) : launch_grid(one, grid, block, 0, s, launch_overlap(), a);
}

}  // namespace

cudaError_t launch_kv4_write(const KvRowsArgs& a, int dtype, cudaStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        return launch_rows<kTokens<T>>(a, s, kv4_write_kernel<T, 1>, kv4_write_kernel<T, kTokens<T>>);
    });
}

cudaError_t launch_kv4_read(const KvRowsArgs& a, int dtype, cudaStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        return launch_rows<kTokens<T>>(a, s, kv4_read_kernel<T, 1>, kv4_read_kernel<T, kTokens<T>>);
    });
}

}  // namespace q4
