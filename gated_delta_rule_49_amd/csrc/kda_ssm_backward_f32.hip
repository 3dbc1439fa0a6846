// Gradients of the state space scan, fp32 inputs.
#include "kda_ssm_backward.hpp"

namespace kda {
hipError_t ssm_grad_f32(const SsmGrad &a, hipStream_t s) { return grad_n<float>(a, s); }
}  // namespace kda
