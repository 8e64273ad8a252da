// Down projections of a mixture of experts: see moe_experts.cuh.
#include "moe_experts.cuh"

namespace q4 {

cudaError_t launch_moe_down_products(const ExpertParams& p, const DeviceInfo& di, cudaStream_t s) {
    return launch_experts_of<false, 2>(p, di, true, s);
}

}  // namespace q4
