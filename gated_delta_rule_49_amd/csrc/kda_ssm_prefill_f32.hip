// fp32 inputs of the state space scan.
#include "kda_ssm_prefill.hpp"

namespace kda {

hipError_t ssm_phase_f32(const SsmScan &q, const SsmPlan &plan, int phase, int out_dtype, hipStream_t s) {
    if (out_dtype == 0) return ssm_phase<float, float>(q, plan, phase, s);
    return ssm_phase<float, bf16_t>(q, plan, phase, s);
}
hipError_t ssm_states_f32(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int phase, hipStream_t s) {
    return ssm_states<float>(f, r, plan, phase, s);
}

}  // namespace kda
