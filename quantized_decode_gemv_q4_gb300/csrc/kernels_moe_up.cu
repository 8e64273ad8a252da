// Gate and up projections of a mixture-of-experts layer, with SwiGLU: see moe_experts.cuh.
#include "moe_experts.cuh"

namespace q4 {

cudaError_t launch_moe_gate_up(const ExpertParams& p, bool bf16_values, const DeviceInfo& di, cudaStream_t s) {
    return bf16_values ? launch_experts_of<true, 1>(p, di, true, s) : launch_experts_of<true, 2>(p, di, true, s);
}

}  // namespace q4
