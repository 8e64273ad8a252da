// RMSNorm of every query and key head and the rotary rotation of its first `rot` elements, in one pass.
//
//   y_i = x_i * r * gamma_i, r = 1 / sqrt(sum x^2 / D + eps);   a pair (a, b) of y turns to
//   (a cos - b sin, b cos + a sin) with the cos and sin of the token's position from a table.
//
// A group of lanes holds one head row: each lane two 16-byte vectors that contain both elements of its pairs (for the
// half-split order vectors rot/2 apart, for the interleaved order adjacent ones; behind the rotated part adjacent
// vectors pass unrotated), so the rotation needs no exchange and the only shuffles are the norm's sum. Sums and
// products are fp32, and the values are rounded once, when they are stored. A row is read whole before it is written,
// so the outputs may be the inputs.
#include "kv_common.cuh"

namespace q4 {

namespace {

constexpr int kThreads = 256;

template <typename T, int LPR>  // LPR: lanes per head row
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs p) {
    constexpr int V = Vec<T>::N;
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = blockIdx.x;
    const int lane = threadIdx.x % LPR;
    const int row = (int)blockIdx.y * (kThreads / LPR) + threadIdx.x / LPR;  // query heads, then key heads
    const bool is_q = row < p.Hq;
    const int pairs = p.rot / (2 * V);  // slots of two vectors that are rotated
    const bool active = row < p.Hq + p.Hkv && lane < p.D / (2 * V);
    const bool turns = lane < pairs;
    const int ia = turns && !p.interleaved ? lane * V : 2 * lane * V;
    const int ib = turns && !p.interleaved ? p.rot / 2 + lane * V : ia + V;
    const int head = is_q ? row : row - p.Hq;
    const T* src = is_q ? static_cast<const T*>(p.q) + t * p.q_stride : static_cast<const T*>(p.k) + t * p.k_stride;
    T* dst = is_q ? static_cast<T*>(p.q_out) + t * p.q_out_stride : static_cast<T*>(p.k_out) + t * p.k_out_stride;
    src += (long long)head * p.D;
    dst += (long long)head * p.D;
    const float* gamma = is_q ? p.q_gamma : p.k_gamma;

    float a[V] = {}, b[V] = {}, c[V] = {}, s[V] = {};
    bool bad = false;
    if (active) {
        load_floats(src + ia, a);
        load_floats(src + ib, b);
        if (pairs > 0) {
            const int pos = p.positions[t];
            bad = pos < 0 || pos >= p.max_pos;
            if (turns && !bad) {
                const float* table = p.cos_sin + (long long)pos * p.rot + lane * V;
                load_floats(table, c);
                load_floats(table + p.rot / 2, s);
            }
        }
    }
    if (gamma) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(sum / (float)p.D + p.eps);
        if (active) {
            float ga[V], gb[V];
            load_floats(gamma + ia, ga);
            load_floats(gamma + ib, gb);
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] = a[i] * r * ga[i], b[i] = b[i] * r * gb[i];
        }
    }
    if (!active) return;
    float oa[V], ob[V];
    if (p.interleaved && turns) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            oa[i] = a[i] * c[i / 2] - a[i + 1] * s[i / 2];
            oa[i + 1] = a[i + 1] * c[i / 2] + a[i] * s[i / 2];
            ob[i] = b[i] * c[(V + i) / 2] - b[i + 1] * s[(V + i) / 2];
            ob[i + 1] = b[i + 1] * c[(V + i) / 2] + b[i] * s[(V + i) / 2];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            oa[i] = turns ? a[i] * c[i] - b[i] * s[i] : a[i];
            ob[i] = turns ? b[i] * c[i] + a[i] * s[i] : b[i];
        }
    }
    if (bad) {  // no table row: the token's heads are NaN
#pragma unroll
        for (int i = 0; i < V; ++i) oa[i] = ob[i] = qnan();
        if (lane == 0) atomicOr(p.fault, (unsigned)kFaultBadPosition);
    }
    store_floats(dst + ia, oa);
    store_floats(dst + ib, ob);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, int dtype, cudaStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        const int slots = a.D / (2 * Vec<T>::N);
        auto go = [&](auto lpr) {
            constexpr int LPR = decltype(lpr)::value;
            const int rows = kThreads / LPR;
            const dim3 grid((unsigned)a.T, (unsigned)((a.Hq + a.Hkv + rows - 1) / rows));
            return launch_grid(qk_norm_rope_kernel<T, LPR>, grid, dim3(kThreads), 0, s, launch_overlap(), a);
        };
        if (slots <= 4) return go(std::integral_constant<int, 4>());
        if (slots <= 8) return go(std::integral_constant<int, 8>());
        if (slots <= 16) return go(std::integral_constant<int, 16>());
        return go(std::integral_constant<int, 32>());
    });
}

}  // namespace q4
