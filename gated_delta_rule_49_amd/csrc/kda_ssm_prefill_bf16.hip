// bf16 inputs of the state space scan.
#include "kda_ssm_prefill.hpp"

namespace kda {

hipError_t ssm_phase_f32(const SsmScan &q, const SsmPlan &plan, int phase, int out_dtype, hipStream_t s);
hipError_t ssm_states_f32(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int phase, hipStream_t s);

hipError_t launch_ssm_phase(const SsmScan &q, const SsmPlan &plan, int phase, int in_dtype, int out_dtype, hipStream_t s) {
    if (in_dtype == 0) return ssm_phase_f32(q, plan, phase, out_dtype, s);
    if (out_dtype == 0) return ssm_phase<bf16_t, float>(q, plan, phase, s);
    return ssm_phase<bf16_t, bf16_t>(q, plan, phase, s);
}
hipError_t launch_ssm_states(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int phase, int in_dtype, hipStream_t s) {
    return in_dtype == 0 ? ssm_states_f32(f, r, plan, phase, s) : ssm_states<bf16_t>(f, r, plan, phase, s);
}

}  // namespace kda
