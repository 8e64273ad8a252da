// The norm behind a block, its gate and scales, the residual sum and the norm before the next block, in one pass.
//
//   b = x, or x * r(x) * post_gamma;  h = residual_scale * residual + branch_scale * gate * b;
//   y = h * r(h) * pre_gamma;         r(v) = 1 / sqrt(sum v^2 / K + eps).
//
// A group of P threads holds a row in registers, V = 16 bytes of activations (VPT times) a thread, so every input is read
// once and every output written once; the two sums of squares meet in shuffles and, where a row has more than one warp, in
// shared memory. Everything between the loads and the stores is fp32: y follows from the fp32 h, not from the stored one.
// A thread reads its elements of x and residual before it writes any of them, so the outputs may be these inputs.
//
// Long prompts are bound by memory: 8191 bf16 rows of 4096 take 48 us, 5.6 TB/s of two reads and two writes, 0.82 of what a
// copy (one of each) reaches. Few rows are bound by the launch and two chains of load, sum and store: 1.9 us for one.
#include <algorithm>

#include "block.h"
#include "kv_common.cuh"

namespace q4 {

namespace {

// 16 bytes of activations as they lie in memory, and as floats.
__device__ __forceinline__ void widen(uint4 w, float (&x)[4], float) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
}
template <typename T>
__device__ __forceinline__ void widen(uint4 w, float (&x)[8], T tag) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(v[i], tag);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Sum over the P threads of a row, the same bits in each of them. `part` holds a float per warp of the row, and is not
// used again before every thread of the row has read it.
template <int P>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (P > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) part[warp] = v;
        __syncthreads();
        v = lane < P / 32 ? part[lane] : 0.f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

template <typename T, int P, int VPT>
__global__ void __launch_bounds__(P == 32 ? 128 : P) residual_norm_kernel(const ResidualNormArgs p) {
    constexpr int V = Vec<T>::N;
    __shared__ float part[2][32];
    const int at = (P == 32 ? threadIdx.x & 31 : threadIdx.x) * V;
    const long long t = P == 32 ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    const bool row = t < p.T;  // the same for all threads of a row
    grid_dependency_wait();
    grid_launch_dependents();
    if (!row) return;

    const T* x = static_cast<const T*>(p.x) + t * p.x_stride;
    const T* residual = p.residual ? static_cast<const T*>(p.residual) + t * p.residual_stride : nullptr;
    const T* gate = p.gate ? static_cast<const T*>(p.gate) + t * p.gate_stride : nullptr;
    constexpr bool kGateEarly = VPT < 8;  // eight vectors leave no registers for the gate's
    uint4 wx[VPT], wr[VPT], wg[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = at + i * P * V;
        wx[i] = wr[i] = wg[i] = make_uint4(0u, 0u, 0u, 0u);
        if (k < p.K) {
            wx[i] = __ldcs(reinterpret_cast<const uint4*>(x + k));
            if (residual) wr[i] = __ldcs(reinterpret_cast<const uint4*>(residual + k));
            if (kGateEarly && gate && p.gate_width > 1) wg[i] = *reinterpret_cast<const uint4*>(gate + k);
        }
    }
    float scale = p.branch_scale;
    if (gate && p.gate_width == 1) scale *= to_float(*gate);
    float b[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i) widen(wx[i], b[i], T());
    if (p.post_gamma) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(b[i][j], b[i][j], sum);
        const float r = rsqrtf(row_sum<P>(sum, part[0]) / (float)p.K + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = at + i * P * V;
            float g[V] = {};
            if (k < p.K) load_floats(p.post_gamma + k, g);
#pragma unroll
            for (int j = 0; j < V; ++j) b[i][j] = b[i][j] * r * g[j];
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = at + i * P * V;
        if (gate && p.gate_width > 1) {
            if (!kGateEarly && k < p.K) wg[i] = *reinterpret_cast<const uint4*>(gate + k);
            float g[V];
            widen(wg[i], g, T());
#pragma unroll
            for (int j = 0; j < V; ++j) b[i][j] *= g[j];
        }
        float r[V];
        widen(wr[i], r, T());
#pragma unroll
        for (int j = 0; j < V; ++j) {
            b[i][j] = residual ? fmaf(p.residual_scale, r[j], scale * b[i][j]) : scale * b[i][j];
            if (k < p.K) sum = fmaf(b[i][j], b[i][j], sum);
        }
        if (k < p.K) store_floats(static_cast<T*>(p.h_out) + t * p.h_stride + k, b[i]);
    }
    if (!p.y_out) return;
    const float r = rsqrtf(row_sum<P>(sum, part[1]) / (float)p.K + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = at + i * P * V;
        if (k >= p.K) continue;
        float g[V];
        load_floats(p.pre_gamma + k, g);
#pragma unroll
        for (int j = 0; j < V; ++j) b[i][j] = b[i][j] * r * g[j];
        store_floats(static_cast<T*>(p.y_out) + t * p.y_stride + k, b[i]);
    }
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs& a, int dtype, cudaStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        const int vecs = (a.K + Vec<T>::N - 1) / Vec<T>::N;
        // launched ahead whatever the overlap setting: the kernel touches nothing before it has waited
        auto go = [&](auto threads, auto vpt) {
            constexpr int P = decltype(threads)::value, VPT = decltype(vpt)::value;
            const dim3 grid((unsigned)(P == 32 ? (a.T - 1) / 4 + 1 : a.T)), block(P == 32 ? 128 : P);
            return launch_grid(residual_norm_kernel<T, P, VPT>, grid, block, 0, s, true, a);
        };
        auto threads = [&](int vpt) { return (vecs + vpt - 1) / vpt; };
        constexpr auto one = std::integral_constant<int, 1>();
        constexpr auto two = std::integral_constant<int, 2>();
        constexpr auto four = std::integral_constant<int, 4>();
        constexpr auto eight = std::integral_constant<int, 8>();
        if (threads(1) <= 32) return go(std::integral_constant<int, 32>(), one);
        // Where several rows wait for each SM, more loads of a thread are worth more than more threads of a row: 8191 bf16 rows
        // of 4096 49.7 us with two vectors a thread, 48.1 us with four (39.6 us for the bytes; 0.82 of the copy rate), 50.4 us
        // with eight. Resident CTAs that walk over the rows and load one ahead: 47.7 us, but 3.3 us instead of 2.9 for 67 rows.
        if (a.T >= 8LL * a.sm_count) {
            if (threads(4) > 64 && threads(4) <= 128) return go(std::integral_constant<int, 128>(), four);
            if (threads(4) > 128 && threads(4) <= 256) return go(std::integral_constant<int, 256>(), four);
            if (threads(4) > 256 && threads(4) <= 512) return go(std::integral_constant<int, 512>(), four);
        }
        if (threads(2) <= 128) return go(std::integral_constant<int, 128>(), two);
        if (threads(2) <= 256) return go(std::integral_constant<int, 256>(), two);
        if (threads(2) <= 512) return go(std::integral_constant<int, 512>(), two);
        if (threads(4) <= 512) return go(std::integral_constant<int, 512>(), four);
        if constexpr (sizeof(T) == 4) {
            // Its 64 registers a thread do not hold a row: 460 bytes of spills. 512 rows of 32768 take 80 us, 40 us for the bytes.
            if (threads(8) > 512) return go(std::integral_constant<int, 1024>(), eight);
        }
        return go(std::integral_constant<int, 512>(), eight);
    });
}

}  // namespace q4
