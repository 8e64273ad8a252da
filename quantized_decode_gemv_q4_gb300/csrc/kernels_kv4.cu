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

// One thread holds 8 elements, four threads a block; the threads of a token run over its K heads, then its V heads.
template <typename T>
__global__ void kv4_write_kernel(const KvRowsArgs p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = (int)blockIdx.x * blockDim.y + threadIdx.y;
    const int per = p.c.num_kv_heads * p.c.head_dim / 8;  // threads' worth of work in K, and in V
    int slot = -1;
    if (t < p.T) slot = p.slots[t];
    if (slot >= p.c.num_pages * p.c.page_size) {
        if (threadIdx.x == 0) atomicOr(p.fault, (unsigned)kFaultBadSlot);
        slot = -1;
    }
    const int page = slot / p.c.page_size, off = slot - page * p.c.page_size;
    const int rounds = (2 * per + (int)blockDim.x - 1) / (int)blockDim.x;
    for (int i = 0; i < rounds; ++i) {  // every thread of a warp takes part in the shuffles
        const int u = i * (int)blockDim.x + threadIdx.x;
        const bool active = slot >= 0 && u < 2 * per;
        const bool is_v = u >= per;
        const int el = (is_v ? u - per : u) * 8;
        float x[8] = {};
        if (active) {
            const T* src = is_v ? static_cast<const T*>(p.v) + t * p.v_stride : static_cast<const T*>(p.k) + t * p.k_stride;
            load_floats(src + el, x);
        }
        uint32_t top = 0u;  // the largest magnitude's bits: NaN and infinity rank above every finite value
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const __half dh = __float2half_rn(fminf(__fdiv_rn(__uint_as_float(top), 7.f), 65504.f));
        const float d = __half2float(dh);
        const bool finite = top < 0x7F800000u;
        const bool codes = finite && d > 0.f;
        const float inv = 1.f / d;
        uint32_t w[2] = {0x08080808u, 0x08080808u};
        if (codes) {
            w[0] = w[1] = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j / 4] |= (uint32_t)(8 + __float2int_rn(nearest_quotient(x[j], d, inv))) << (8 * (j % 4));
        }
        // thread q of a block holds elements 8q .. 8q + 7: bytes 8 (q % 2) .. + 7, low nibbles from q < 2
        const int q = threadIdx.x & 3;
        const uint32_t o0 = __shfl_xor_sync(0xffffffffu, w[0], 2), o1 = __shfl_xor_sync(0xffffffffu, w[1], 2);
        const uint32_t word = q < 2 ? (w[0] | (o0 << 4)) : (o1 | (w[1] << 4));
        if (active) {
            const int h = el / p.c.head_dim, in_row = el - h * p.c.head_dim;
            const long long row = cache_row(p.c, page, h, off);
            uint8_t* qs = (is_v ? p.c.v_qs : p.c.k_qs) + row * (p.c.head_dim / 2);
            uint16_t* ds = (is_v ? p.c.v_d : p.c.k_d) + row * (p.c.head_dim / 32);
            *reinterpret_cast<uint32_t*>(qs + (in_row / 32) * 16 + (q & 1) * 8 + (q >> 1) * 4) = word;
            if (q == 0) ds[in_row / 32] = finite ? __half_as_ushort(dh) : (unsigned short)0x7E00u;
        }
    }
}

template <typename T>
__global__ void kv4_read_kernel(const KvRowsArgs p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = (int)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.T) return;
    const int per = p.c.num_kv_heads * p.c.head_dim / 8;
    const int slot = p.slots[t];
    if (slot < 0) return;
    const bool bad = slot >= p.c.num_pages * p.c.page_size;
    if (bad && threadIdx.x == 0) atomicOr(p.fault, (unsigned)kFaultBadSlot);
    const int page = bad ? 0 : slot / p.c.page_size, off = bad ? 0 : slot - page * p.c.page_size;
    for (int u = threadIdx.x; u < 2 * per; u += blockDim.x) {
        const bool is_v = u >= per;
        const int el = (is_v ? u - per : u) * 8;
        T* dst = static_cast<T*>(is_v ? p.v : p.k);
        if (!dst) continue;
        dst += t * (is_v ? p.v_stride : p.k_stride) + el;
        const int h = el / p.c.head_dim, in_row = el - h * p.c.head_dim;
        const long long row = cache_row(p.c, page, h, off);
        const int q = (in_row / 8) & 3;
        const uint2 w = *reinterpret_cast<const uint2*>((is_v ? p.c.v_qs : p.c.k_qs) + row * (p.c.head_dim / 2) +
                                                        (in_row / 32) * 16 + (q & 1) * 8);
        float d = f16_bits_to_f32((is_v ? p.c.v_d : p.c.k_d)[row * (p.c.head_dim / 32) + in_row / 32]);
        if (bad) d = qnan();
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t code = ((j < 4 ? w.x : w.y) >> (8 * (j % 4) + 4 * (q >> 1))) & 15u;
            x[j] = (float)((int)code - 8) * d;
        }
        store_floats(dst, x);
    }
}

// A block's threads: x over a token's 2 * Hkv * D / 8 eight-element pieces (a multiple of 8), y over tokens so that
// short tokens share a block; a whole number of warps.
dim3 rows_block(const KvRowsArgs& a) {
    const int pieces = 2 * a.c.num_kv_heads * a.c.head_dim / 8;
    if (pieces >= kThreads) return dim3(kThreads);
    int y = kThreads / pieces;
    if (pieces % 32) y = (y + 3) / 4 * 4;
    return dim3((unsigned)pieces, (unsigned)y);
}

}  // namespace

cudaError_t launch_kv4_write(const KvRowsArgs& a, int dtype, cudaStream_t s) {
    const dim3 block = rows_block(a);
    const dim3 grid((unsigned)((a.T + (int)block.y - 1) / (int)block.y));
    return with_dtype(dtype, [&](auto tag) {
        return launch_grid(kv4_write_kernel<decltype(tag)>, grid, block, 0, s, launch_overlap(), a);
    });
}

cudaError_t launch_kv4_read(const KvRowsArgs& a, int dtype, cudaStream_t s) {
    const dim3 block = rows_block(a);
    const dim3 grid((unsigned)((a.T + (int)block.y - 1) / (int)block.y));
    return with_dtype(dtype, [&](auto tag) {
        return launch_grid(kv4_read_kernel<decltype(tag)>, grid, block, 0, s, launch_overlap(), a);
    });
}

}  // namespace q4
