// bf16 inputs of the state space scan.
#include "kda_ssm_prefill.hpp"

namespace kda {

hipError_t ssm_phase_f32(const SsmScan &q, const SsmPlan &plan, int mode, int phase, int out_dtype, hipStream_t s);

hipError_t launch_ssm_phase(const SsmScan &q, const SsmPlan &plan, int mode, int phase, int in_dtype, int out_dtype, hipStream_t s) {
    if (in_dtype == 0) return ssm_phase_f32(q, plan, mode, phase, out_dtype, s);
    if (out_dtype == 0) return ssm_phase<bf16_t, float>(q, plan, mode, phase, s);
    return ssm_phase<bf16_t, bf16_t>(q, plan, mode, phase, s);
}

}  // namespace kda
