// A whole mixture-of-experts layer for a few tokens over planar Q4 experts, and its last part alone (the experts' down
// projections and their weighted sum).
//
//   xn = x, or x * r * gamma;  logits = Wr xn, top-k and softmax weights (the router's kernel);
//   h[t, s] = silu(Wg xn) * (Wu xn) and z[t, s] = Wd h[t, s] of expert e(t, s);
//   out[t] = residual[t] + sum over s of weight[t, s] * z[t, s].
//
// Four kernels for a layer: the router (kernels_router.cu), gate and up, down (moe_experts.cuh) and the join here; three for the
// down projections alone, whose first takes the largest size of each slot's vector, which gate and up leaves by itself. Each may
// start while the one before it ends (programmatic dependent launch) and waits for it before it touches what it wrote. A call's
// first kernel is launched so whatever the overlap setting (1 token 29.7 us a call, 27.8 us so): with the setting off it touches
// nothing before it has waited, with it on the layer's router reads some of its weights. h, z, the picks and xn stay in the workspace.
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

// The largest size in each row of [rows][cols], as its bits.
__global__ void __launch_bounds__(256) moe_max_kernel(const float* x, unsigned* out, int cols) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ unsigned part[8];
    const float* row = x + (long long)blockIdx.x * cols;
    unsigned m = 0u;
    for (int k = threadIdx.x * 4; k < cols; k += 1024) {
        float v[4];
        load_floats(row + k, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, part[i]);
        out[blockIdx.x] = m;
    }
}

struct JoinParams {
    void* out;
    const void* residual;
    const float *z, *weights;
    const int32_t* ids;
    int topk, E, rows, parts, slots;
    long long out_stride, residual_stride;
    int32_t* status;
    unsigned* fault;
};

// out[t] = residual[t] + sum_s weights[t][s] * z[t][s], in the order of the slots. The picks and the residual were written
// before the kernel before this one began, so they are read while it runs.
template <typename T>
__global__ void __launch_bounds__(128) moe_join_kernel(const JoinParams p) {
    const int t = blockIdx.y, n = (blockIdx.x * 128 + threadIdx.x) * 4;
    const bool in = n < p.rows;
    constexpr int kAtOnce = 8;
    int e[kAtOnce];
    float w[kAtOnce];
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s) {
        const bool there = in && s < p.topk;
        e[s] = there ? __ldcg(p.ids + t * p.topk + s) : 0;
        w[s] = there ? __ldcg(p.weights + t * p.topk + s) : 0.f;
    }
    float v[4] = {};
    if (in && p.residual) {
        const T* r = static_cast<const T*>(p.residual) + t * p.residual_stride + n;
        if constexpr (sizeof(T) == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(r));
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
            const uint2 u = __ldcg(reinterpret_cast<const uint2*>(r));
            const float2 a = unpack2(u.x, T()), b = unpack2(u.y, T());
            v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        }
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (!in) return;
    bool bad = false;
    auto add = [&](int s, int e, float w) {
        if (e < 0 || e >= p.E) {
            bad = true;
            return;
        }
        const float* from = p.z + ((long long)t * p.topk + s) * p.rows + n;
        float z[4];
        load_floats(from, z);
        for (int q = 1; q < p.parts; ++q) {
            float more[4];
            load_floats(from + (long long)q * p.slots * p.rows, more);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] += more[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(w, z[j], v[j]);
    };
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s)
        if (s < p.topk) add(s, e[s], w[s]);
    for (int s = kAtOnce; s < p.topk; ++s) add(s, p.ids[t * p.topk + s], p.weights[t * p.topk + s]);
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
    unsigned* h_max;
    DownSpace(Carve& c, int slots, int rows, int cols)
        : z(c.take<float>((size_t)moe_parts(cols / 32) * slots * rows)), h_max(c.take<unsigned>(slots)) {}
};

cudaError_t launch_down(const DownSpace& w, const float* h, const uint8_t* qs, const uint16_t* d, const int32_t* ids, int slots,
                        int E, int rows, int cols, const DeviceInfo& di, cudaStream_t s) {
    ExpertParams p = {};
    p.qs0 = p.qs1 = qs, p.d0 = p.d1 = d;
    p.in = h, p.in_max = w.h_max, p.out = w.z, p.ids = ids;
    p.E = E, p.rows = rows, p.blocks = cols / 32, p.slots = slots, p.per_in = 1;
    return launch_moe_down_products(p, di, s);
}

}  // namespace

size_t moe_down_workspace_bytes(int T, int topk, int rows, int cols) {
    Carve c{nullptr};
    DownSpace(c, T * topk, rows, cols);
    return c.at;
}

cudaError_t launch_moe_down(const MoeDownArgs& a, int dtype, void* workspace, const DeviceInfo& di, cudaStream_t s) {
    Carve c{static_cast<uint8_t*>(workspace)};
    const int slots = a.T * a.topk;
    const DownSpace w(c, slots, a.rows, a.cols);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)slots), cfg.blockDim = dim3(256), cfg.stream = s;
    cfg.attrs = attr, cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, moe_max_kernel, a.h, w.h_max, a.cols);
    if (e != cudaSuccess) return e;
    if ((e = launch_down(w, a.h, a.qs, a.d, a.ids, slots, a.E, a.rows, a.cols, di, s)) != cudaSuccess) return e;
    const JoinParams join = {a.out, a.residual, w.z, a.weights, a.ids, a.topk, a.E, a.rows, moe_parts(a.cols / 32), slots,
                             a.out_stride, a.residual_stride, a.status, a.fault};
    return launch_join(join, a.T, dtype, true, s);
}

struct LayerSpace {
    float *xn, *h, *weights;
    int32_t* ids;
    unsigned* x_max;
    DownSpace down;
    LayerSpace(Carve& c, int T, int topk, int N, int K)
        : xn(c.take<float>((size_t)T * K)), h(c.take<float>((size_t)T * topk * N)), weights(c.take<float>(T * topk)),
          ids(c.take<int32_t>(T * topk)), x_max(c.take<unsigned>(T)), down(c, T * topk, K, N) {}
};

size_t moe_layer_workspace_bytes(int T, int topk, int N, int K) {
    Carve c{nullptr};
    LayerSpace(c, T, topk, N, K);
    return c.at;
}

cudaError_t launch_moe_layer(const MoeLayerArgs& a, int dtype, void* workspace, const DeviceInfo& di, cudaStream_t s) {
    Carve c{static_cast<uint8_t*>(workspace)};
    const int slots = a.T * a.topk, N = a.w.N, K = a.w.K, E = a.w.E;
    const LayerSpace w(c, a.T, a.topk, N, K);
    int32_t* ids = a.ids ? a.ids : w.ids;
    float* weights = a.weights ? a.weights : w.weights;
    const LayerInput in = {a.x, a.gamma, w.xn, w.x_max, w.down.h_max, a.eps, a.x_stride, launch_overlap()};
    cudaError_t e = launch_moe_layer_router(ids, weights, a.w.router_qs, a.w.router_d, in, dtype, a.T, E, K, a.topk,
                                            a.normalize != 0, s);
    if (e != cudaSuccess) return e;
    ExpertParams up = {};
    up.qs0 = a.w.gate_qs, up.qs1 = a.w.up_qs, up.d0 = a.w.gate_d, up.d1 = a.w.up_d;
    up.in = w.xn, up.in_max = w.x_max, up.out = w.h, up.out_max = w.down.h_max, up.ids = ids;
    up.E = E, up.rows = N, up.blocks = K / 32, up.slots = slots, up.per_in = a.topk;
    if ((e = launch_moe_gate_up(up, dtype == Q4_BF16 && !a.gamma, di, s)) != cudaSuccess) return e;
    if ((e = launch_down(w.down, w.h, a.w.down_qs, a.w.down_d, ids, slots, E, K, N, di, s)) != cudaSuccess) return e;
    const JoinParams join = {a.out, a.residual, w.down.z, weights, ids, a.topk, E, K, moe_parts(N / 32), slots, a.out_stride,
                             a.residual_stride, nullptr, a.fault};
    return launch_join(join, a.T, dtype, true, s);
}

}  // namespace q4
