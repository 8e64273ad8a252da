// Gate and up projections of a mixture-of-experts layer, with SwiGLU: see moe_experts.cuh.
#include "moe_experts.cuh"

namespace q4 {

cudaError_t launch_moe_gate_up(const ExpertParams& p, int dtype, const DeviceInfo& di, cudaStream_t s) {
    return launch_experts<true>(p, dtype, di, true, s);
}

}  // namespace q4
