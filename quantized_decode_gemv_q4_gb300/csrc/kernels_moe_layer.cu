// A whole mixture-of-experts layer for a few tokens over planar Q4 experts, and its last part alone (the experts' down
// projections and their weighted sum).
//
//   xn = x, or x * r * gamma;  logits = Wr xn, top-k and softmax weights (the router's kernel);
//   h[t, s] = silu(Wg xn) * (Wu xn) and z[t, s] = Wd h[t, s] of expert e(t, s);
//   out[t] = residual[t] + sum over s of weight[t, s] * z[t, s].
#include <algorithm>

#include "block.h"
#include "kv_common.cuh"

namespace q4 {

namespace {

struct Carve {  // parts of a workspace, each 16-byte aligned
    uint8_t* base;
    size_t at = 0;
    template <typename T>
    T* take(size_t n) {
        T* p = reinterpret_cast<T*>(base + at);
        at += (n * sizeof(T) + 15) / 16 * 16;
        return base ? p : nullptr;
    }
};

struct PrepParams {
    const void* x;
    const float* gamma;
    float* xn;
    float eps;
    int K;
    long long x_stride;
};

// xn[t] = x[t], or its norm, in fp32.
template <typename T>
__global__ void __launch_bounds__(256) moe_prep_kernel(const PrepParams p) {
    constexpr int V = Vec<T>::N;
    __shared__ float part[8];
    const T* x = static_cast<const T*>(p.x) + (long long)blockIdx.x * p.x_stride;
    float* xn = p.xn + (long long)blockIdx.x * p.K;
    grid_dependency_wait();
    grid_launch_dependents();
    float r = 1.f;
    if (p.gamma) {
        float sum = 0.f;
        for (int k = threadIdx.x * V; k < p.K; k += 256 * V) {
            float v[V];
            load_floats(x + k, v);
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(v[j], v[j], sum);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += part[i];
        r = rsqrtf(sum / (float)p.K + p.eps);
    }
    for (int k = threadIdx.x * V; k < p.K; k += 256 * V) {
        float v[V];
        load_floats(x + k, v);
        if (p.gamma) {
            float g[V];
            load_floats(p.gamma + k, g);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = v[j] * r * g[j];
        }
        store_floats(xn + k, v);
    }
}

struct ExpertParams {
    const uint8_t *qs0, *qs1;  // one matrix (down), or gate and up
    const uint16_t *d0, *d1;
    const float* in;
    float* out;  // [slots][rows]
    const int32_t* ids;
    int E, rows, cols, per_in;  // slot s reads input row s / per_in
};

__device__ __forceinline__ float block_dot(const uint8_t* qs, float d, const float* x) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int b = qs[j];
        sum = fmaf((float)((b & 15) - 8), x[j], sum);
        sum = fmaf((float)((b >> 4) - 8), x[j + 16], sum);
    }
    return sum * d;
}

// A warp per (slot, row).
template <bool GateUp>
__global__ void __launch_bounds__(256) moe_expert_kernel(const ExpertParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31, slot = blockIdx.y;
    const int e = p.ids[slot];
    if (row >= p.rows || e < 0 || e >= p.E) return;
    const int blocks = p.cols / 32;
    const long long first = ((long long)e * p.rows + row) * blocks;
    const float* x = p.in + (long long)(slot / p.per_in) * p.cols;
    float a = 0.f, b = 0.f;
    for (int i = lane; i < blocks; i += 32) {
        a += block_dot(p.qs0 + (first + i) * 16, f16_bits_to_f32(p.d0[first + i]), x + i * 32);
        if (GateUp) b += block_dot(p.qs1 + (first + i) * 16, f16_bits_to_f32(p.d1[first + i]), x + i * 32);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane == 0) p.out[(long long)slot * p.rows + row] = GateUp ? silu(a) * b : a;
}

struct JoinParams {
    void* out;
    const void* residual;
    const float *z, *weights;
    const int32_t* ids;
    int topk, E, rows;
    long long out_stride, residual_stride;
    int32_t* status;
    unsigned* fault;
};

// out[t] = residual[t] + sum_s weights[t][s] * z[t][s], in the order of the slots.
template <typename T>
__global__ void __launch_bounds__(128) moe_join_kernel(const JoinParams p) {
    const int t = blockIdx.y, n = (blockIdx.x * 128 + threadIdx.x) * 4;
    grid_dependency_wait();
    grid_launch_dependents();
    if (n >= p.rows) return;
    float v[4] = {};
    if (p.residual) {
        const T* r = static_cast<const T*>(p.residual) + t * p.residual_stride + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)r[j];
    }
    bool bad = false;
    for (int s = 0; s < p.topk; ++s) {
        const long long slot = (long long)t * p.topk + s;
        const int e = p.ids[slot];
        if (e < 0 || e >= p.E) {
            bad = true;
            continue;
        }
        const float w = p.weights[slot];
        float z[4];
        load_floats(p.z + slot * p.rows + n, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(w, z[j], v[j]);
    }
    if (bad) {  // an expert that is not there: the token's row is NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = qnan();
        if (n == 0) {
            if (p.status) *p.status = (int32_t)kFaultBadExpert;
            atomicOr(p.fault, (unsigned)kFaultBadExpert);
        }
    }
    T* out = static_cast<T*>(p.out) + t * p.out_stride + n;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()));
    }
}

cudaError_t launch_join(const JoinParams& p, int T, int dtype, bool overlap, cudaStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        const dim3 grid((unsigned)((p.rows + 511) / 512), (unsigned)T);
        return launch_grid(moe_join_kernel<decltype(tag)>, grid, dim3(128), 0, s, overlap, p);
    });
}

struct DownSpace {
    float* z;
    DownSpace(Carve& c, int slots, int rows, int) { z = c.take<float>((size_t)slots * rows); }
};

}  // namespace

size_t moe_down_workspace_bytes(int T, int topk, int rows, int cols) {
    Carve c{nullptr};
    DownSpace(c, T * topk, rows, cols);
    return c.at;
}

cudaError_t launch_moe_down(const MoeDownArgs& a, int dtype, void* workspace, const DeviceInfo&, cudaStream_t s) {
    Carve c{static_cast<uint8_t*>(workspace)};
    const int slots = a.T * a.topk;
    const DownSpace w(c, slots, a.rows, a.cols);
    const ExpertParams down = {a.qs, nullptr, a.d, nullptr, a.h, w.z, a.ids, a.E, a.rows, a.cols, 1};
    cudaError_t e = launch_grid(moe_expert_kernel<false>, dim3((unsigned)((a.rows + 7) / 8), (unsigned)slots), dim3(256), 0, s,
                                launch_overlap(), down);
    if (e != cudaSuccess) return e;
    const JoinParams join = {a.out, a.residual, w.z, a.weights, a.ids, a.topk, a.E, a.rows, a.out_stride, a.residual_stride,
                             a.status, a.fault};
    return launch_join(join, a.T, dtype, true, s);
}

struct LayerSpace {
    float *xn, *h, *weights;
    int32_t* ids;
    DownSpace down;
    LayerSpace(Carve& c, int T, int topk, int N, int K)
        : xn(c.take<float>((size_t)T * K)), h(c.take<float>((size_t)T * topk * N)), weights(c.take<float>(T * topk)),
          ids(c.take<int32_t>(T * topk)), down(c, T * topk, K, N) {}
};

size_t moe_layer_workspace_bytes(int T, int topk, int N, int K) {
    Carve c{nullptr};
    LayerSpace(c, T, topk, N, K);
    return c.at;
}

cudaError_t launch_moe_layer(const MoeLayerArgs& a, int dtype, void* workspace, const DeviceInfo& di, cudaStream_t s) {
    (void)di;
    Carve c{static_cast<uint8_t*>(workspace)};
    const int slots = a.T * a.topk, N = a.w.N, K = a.w.K, E = a.w.E;
    const LayerSpace w(c, a.T, a.topk, N, K);
    int32_t* ids = a.ids ? a.ids : w.ids;
    float* weights = a.weights ? a.weights : w.weights;
    const PrepParams prep = {a.x, a.gamma, w.xn, a.eps, K, a.x_stride};
    cudaError_t e = with_dtype(dtype, [&](auto tag) {
        return launch_grid(moe_prep_kernel<decltype(tag)>, dim3((unsigned)a.T), dim3(256), 0, s, launch_overlap(), prep);
    });
    if (e != cudaSuccess) return e;
    if ((e = launch_moe_router(ids, weights, nullptr, a.w.router_qs, a.w.router_d, w.xn, a.T, E, K, a.topk, a.normalize != 0,
                               s)) != cudaSuccess)
        return e;
    const ExpertParams up = {a.w.gate_qs, a.w.up_qs, a.w.gate_d, a.w.up_d, w.xn, w.h, ids, E, N, K, a.topk};
    if ((e = launch_grid(moe_expert_kernel<true>, dim3((unsigned)((N + 7) / 8), (unsigned)slots), dim3(256), 0, s, true, up)) !=
        cudaSuccess)
        return e;
    const ExpertParams down = {a.w.down_qs, nullptr, a.w.down_d, nullptr, w.h, w.down.z, ids, E, K, N, 1};
    if ((e = launch_grid(moe_expert_kernel<false>, dim3((unsigned)((K + 7) / 8), (unsigned)slots), dim3(256), 0, s, true, down)) !=
        cudaSuccess)
        return e;
    const JoinParams join = {a.out, a.residual, w.down.z, weights, ids, a.topk, E, K, a.out_stride, a.residual_stride, nullptr,
                             a.fault};
    return launch_join(join, a.T, dtype, true, s);
}

}  // namespace q4
