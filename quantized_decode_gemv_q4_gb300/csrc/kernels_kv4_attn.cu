// Attention of the newest tokens of each sequence over a paged cache held in 4 bits.
//
// Query m of a sequence of length n sits at position p = n - M + m and sees the tokens max(0, p + 1 - window) .. p
// (window 0: all): out = sum_t softmax_t(scale q . k_t) v_t. One CTA per (sequence, query, head): every warp takes
// every fourth token with its own running maximum and sum, and the warps are joined at the end.
#include "kv_common.cuh"

namespace q4 {

namespace {

constexpr int kWarps = 4;

template <typename T, int DB>
__global__ void __launch_bounds__(kWarps * 32) kv4_attention_kernel(const KvAttnArgs p) {
    constexpr int D = DB * 32;
    __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hq = blockIdx.x % p.Hq, bm = blockIdx.x / p.Hq, b = bm / p.M, m = bm % p.M;
    const int h = hq / (p.Hq / p.c.num_kv_heads);
    const int n = p.seq_lens[b];
    bool bad = n < 0 || n > p.max_pages * p.c.page_size;
    if (bad && threadIdx.x == 0) atomicOr(p.fault, (unsigned)kFaultBadLength);
    const int end = bad ? 0 : n - p.M + m + 1;
    const int begin = p.window > 0 ? max(0, end - p.window) : 0;
    const T* q = static_cast<const T*>(p.q) + (long long)bm * p.q_stride + hq * D;
    float qv[DB], o[DB] = {}, mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < DB; ++i) qv[i] = (float)q[32 * i + lane];
    for (int t = begin + warp; t < end; t += kWarps) {
        const int page = p.block_table[(long long)b * p.max_pages + t / p.c.page_size];
        if (page < 0 || page >= p.c.num_pages) {
            if (lane == 0) atomicOr(p.fault, (unsigned)kFaultBadPage);
            bad = true;
            break;
        }
        const long long row = cache_row(p.c, page, h, t % p.c.page_size);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < DB; ++i) {
            const int code = (p.c.k_qs[row * (D / 2) + 16 * i + lane % 16] >> (lane / 16 * 4)) & 15;
            s = fmaf(qv[i], (float)(code - 8) * f16_bits_to_f32(p.c.k_d[row * DB + i]), s);
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale;
        const float nm = fmaxf(mx, s), keep = expf(mx - nm), e = expf(s - nm);
        mx = nm;
        l = l * keep + e;
#pragma unroll
        for (int i = 0; i < DB; ++i) {
            const int code = (p.c.v_qs[row * (D / 2) + 16 * i + lane % 16] >> (lane / 16 * 4)) & 15;
            o[i] = o[i] * keep + e * ((float)(code - 8) * f16_bits_to_f32(p.c.v_d[row * DB + i]));
        }
    }
    if (bad) l = qnan(), mx = 0.f;
#pragma unroll
    for (int i = 0; i < DB; ++i) so[warp][32 * i + lane] = o[i];
    if (lane == 0) sm[warp] = mx, sl[warp] = l;
    __syncthreads();
    float top = -INFINITY, total = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
    const float base = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kWarps; ++w) total += sl[w] * expf(sm[w] - base);
    T* out = static_cast<T*>(p.out) + (long long)bm * p.out_stride + hq * D;
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += so[w][i] * expf(sm[w] - base);
        out[i] = (T)(total == 0.f ? 0.f : v / total);
    }
    if (p.lse && threadIdx.x == 0) p.lse[(long long)bm * p.Hq + hq] = top + logf(total);
}

}  // namespace

size_t kv4_attention_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_kv4_attention(const KvAttnArgs& a, void*, int, cudaStream_t s) {
    return with_dtype(a.dtype, [&](auto tag) {
        using T = decltype(tag);
        const dim3 grid((unsigned)(a.B * a.M * a.Hq));
        auto go = [&](auto db) {
            return launch_grid(kv4_attention_kernel<T, decltype(db)::value>, grid, dim3(kWarps * 32), 0, s,
                               launch_overlap(), a);
        };
        if (a.c.head_dim == 64) return go(std::integral_constant<int, 2>());
        if (a.c.head_dim == 128) return go(std::integral_constant<int, 4>());
        return go(std::integral_constant<int, 8>());
    });
}

}  // namespace q4
