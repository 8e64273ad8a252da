// Internal host-side interface of the block norm and of the mixture-of-experts layer.
// Arguments reaching these functions have already been validated by the ABI layer.
#pragma once

#include "kv.h"
#include "launch.h"

namespace q4 {

struct ResidualNormArgs {
    void *h_out, *y_out;  // y_out nullptr: no norm behind the sum
    const void *x, *residual, *gate;  // residual, gate: nullable
    const float *post_gamma, *pre_gamma;
    float eps, residual_scale, branch_scale;
    int T, K, gate_width;  // gate_width: K (element by element) or 1 (a number per token)
    long long h_stride, y_stride, x_stride, residual_stride, gate_stride;
    int sm_count;
};
cudaError_t launch_residual_norm(const ResidualNormArgs& a, int dtype, cudaStream_t s);

// The experts' products (moe_experts.cuh): gate and up with SwiGLU, or down. The callers fill what comes before `units`.
struct ExpertParams {
    const uint8_t *qs0, *qs1;  // gate and up, or down twice
    const uint16_t *d0, *d1;
    const float* in;
    const unsigned* in_max;    // bits of the largest size in an input row
    float* out;                // [parts][slots][rows]
    unsigned* out_max;         // as in_max, of the outputs (gate and up)
    const int32_t* ids;
    int E, rows, blocks, slots, per_in;  // slot s reads input row s / per_in
    int units, parts, part_blocks, cap, scale_bytes, table_bits;
    uint32_t ring_at, deposits_at, frags_at;
};
// Parts that a down projection's input is cut into (their sums are added by the join), of at most so many blocks: 8 vectors'
// parts fit beside the rings.
constexpr int kPartBlocks = 88;
inline int moe_parts(int blocks) { return (blocks + kPartBlocks - 1) / kPartBlocks; }
// bf16_values: the inputs are bf16 numbers (x as it is), which one f16 part holds.
cudaError_t launch_moe_gate_up(const ExpertParams& p, bool bf16_values, const DeviceInfo& di, cudaStream_t s);
cudaError_t launch_moe_down_products(const ExpertParams& p, const DeviceInfo& di, cudaStream_t s);

// Down projections of T * topk slots and their weighted sum per token: rows = outputs, cols = inputs of an expert's matrix.
struct MoeDownArgs {
    void* out;
    const uint8_t* qs;
    const uint16_t* d;
    const float* h;       // [T][topk][cols]
    const int32_t* ids;   // [T][topk]
    const float* weights; // [T][topk]
    const void* residual; // nullable
    int T, topk, E, rows, cols;
    long long out_stride, residual_stride;
    int32_t* status;  // nullable
    unsigned* fault;
};
size_t moe_down_workspace_bytes(int T, int topk, int rows, int cols);
cudaError_t launch_moe_down(const MoeDownArgs& a, int dtype, void* workspace, const DeviceInfo& di, cudaStream_t s);

struct MoeLayerArgs {
    moe_q4_weights w;
    void* out;
    const void *x, *residual;  // residual: nullable
    const float* gamma;        // nullable: no norm
    float eps;
    int T, topk, normalize;
    long long out_stride, x_stride, residual_stride;
    int32_t* ids;    // nullable (kept in the workspace)
    float* weights;  // nullable
    unsigned* fault;
};

// The layer's input, and what its router's kernel leaves for the experts' kernels.
struct LayerInput {
    const void* x;
    const float* gamma;  // nullable: no norm
    float* xn;           // [T][K]: x or its norm
    unsigned *x_max, *h_max;  // bits of the largest size in a row of xn; zeros for T * topk rows
    float eps;
    long long x_stride;
    bool early;  // router weights may be read before the previous kernel ends (launch overlap is on)
};
cudaError_t launch_moe_layer_router(int32_t* ids, float* weights, const uint8_t* qs, const uint16_t* d, const LayerInput& layer,
                                    int dtype, int T, int E, int K, int topk, bool normalize, cudaStream_t s);

size_t moe_layer_workspace_bytes(int T, int topk, int N, int K);
cudaError_t launch_moe_layer(const MoeLayerArgs& a, int dtype, void* workspace, const DeviceInfo& di, cudaStream_t s);

}  // namespace q4
