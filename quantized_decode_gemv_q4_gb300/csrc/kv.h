// Internal host-side interface of the operators between two projection GEMVs of a decode step: per-head norm with
// rotation, the 4-bit key/value cache and attention over it. Arguments have been validated by the ABI layer.
#pragma once

#include "../../include/q4gemv.h"
#include "launch.h"

namespace q4 {

// As launch_kernel, for a grid and block of several dimensions.
template <typename Kernel, typename Params>
cudaError_t launch_grid(Kernel kern, dim3 grid, dim3 block, uint32_t smem, cudaStream_t s, bool overlap,
                        const Params& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

struct RopeArgs {
    void *q_out, *k_out;
    const void *q, *k;
    const float *q_gamma, *k_gamma, *cos_sin;
    const int32_t* positions;
    float eps;
    int T, Hq, Hkv, D, rot, max_pos, interleaved;
    long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements from one token to the next
    unsigned* fault;
    int sm_count;
};
cudaError_t launch_qk_norm_rope(const RopeArgs& a, int dtype, cudaStream_t s);

struct KvRowsArgs {
    kv4_cache c;
    void *k, *v;  // write: inputs; read: outputs (either may be null when reading)
    const int32_t* slots;
    int T;
    long long k_stride, v_stride;
    unsigned* fault;
    int lp;  // log2(page size)
};
cudaError_t launch_kv4_write(const KvRowsArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_kv4_read(const KvRowsArgs& a, int dtype, cudaStream_t s);

struct KvAttnArgs {
    kv4_cache c;
    void* out;
    float* lse;
    const void* q;
    const int32_t *block_table, *seq_lens;
    int B, M, Hq, max_pages;
    long long q_stride, out_stride;  // elements from one token to the next
    float scale;
    int window;
    int dtype;
    unsigned* fault;
};
// Bytes of workspace that launch_kv4_attention needs for these sizes on a device of sm_count SMs.
size_t kv4_attention_workspace_bytes(int M, int group, int heads, int D, int dtype, int sm_count);
cudaError_t launch_kv4_attention(const KvAttnArgs& a, void* workspace, const DeviceInfo& di, cudaStream_t s);

}  // namespace q4
