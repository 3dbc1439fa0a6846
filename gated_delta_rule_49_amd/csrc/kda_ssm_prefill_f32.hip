// fp32 inputs of the state space scan.
#include "kda_ssm_prefill.hpp"

namespace kda {

hipError_t ssm_phase_f32(const SsmScan &q, const SsmPlan &plan, int mode, int phase, int out_dtype, hipStream_t s) {
    if (out_dtype == 0) return ssm_phase<float, float>(q, plan, mode, phase, s);
    return ssm_phase<float, bf16_t>(q, plan, mode, phase, s);
}

}  // namespace kda
