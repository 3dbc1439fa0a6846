// Gradients of the state space scan: the host side, the sums over the chunks,
// and bf16 inputs (kda_ssm_backward.hpp).
#include "kda_ssm_backward.hpp"

namespace kda {

hipError_t ssm_grad_bf16(const SsmGrad &a, hipStream_t s) { return grad_n<bf16_t>(a, s); }

namespace {
// dA, dD and ddt_bias of a head: its chunks' shares in a fixed order
__global__ void __launch_bounds__(256) ssm_scalar_kernel(SsmGrad a, int64_t items, int sub, float *dA, float *dD, float *dbias) {
    __shared__ double s[4];  // sums of either sign over all chunks: their own rounding would add up
    // without offsets to check, nothing has written the call's status yet
    if (!a.q.p.cu_seqlens && blockIdx.x == 0 && threadIdx.x == 0) *const_cast<int32_t *>(a.q.status) = 0;
    const int which = blockIdx.x / a.q.p.H, h = blockIdx.x % a.q.p.H;
    float *to = which == 0 ? dA : which == 1 ? dD : dbias;
    if (!to || (a.q.p.cu_seqlens && *a.q.status != 0)) return;  // the whole workgroup
    const int64_t n = a.q.p.cu_seqlens ? static_cast<int64_t>(a.q.chunk_off[a.q.p.N]) * sub : items;
    const float *src = a.scalars + (static_cast<int64_t>(which) * a.q.p.H + h) * items;
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 256) v += src[i];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) to[h] = static_cast<float>((s[0] + s[1]) + (s[2] + s[3]));
}
}  // namespace

SsmGradPlan ssm_grad_plan(const SsmParams &p, bool packed, int in_dtype) {
    SsmGradPlan r{};
    r.scan = ssm_plan(p, packed, 2);
    r.sub = in_dtype == 0 ? 2 : 1;
    r.items = r.scan.chunks_bound * r.sub;
    // A block walks several heads of a group, keeping the sums of dB and dC;
    // the group's heads are split over blocks (whose sums another kernel adds)
    // only as far as about 512 blocks need
    const int hpg = p.H / p.G;
    const int64_t per_split = std::max<int64_t>(1, r.items * p.G);
    const int64_t want = std::min<int64_t>(hpg, std::max<int64_t>(1, (512 + per_split - 1) / per_split));
    r.heads_per_block = static_cast<int32_t>((hpg + want - 1) / want);
    r.splits = (hpg + r.heads_per_block - 1) / r.heads_per_block;
    r.state_bytes = align_up(sizeof(float) * static_cast<size_t>(r.items) * p.H * p.Ns * p.P);
    r.scalar_bytes = align_up(sizeof(float) * 3 * static_cast<size_t>(r.items) * p.H);
    if (r.splits > 1) r.part_bytes = align_up(sizeof(float) * r.splits * static_cast<size_t>(p.B) * p.T * p.G * p.Ns);
    return r;
}

hipError_t launch_ssm_backward(const SsmParams &p, const SsmGradOut &o, char *ws, int in_dtype, hipStream_t s) {
    const SsmGradPlan plan = ssm_grad_plan(p, p.cu_seqlens != nullptr, in_dtype);
    SsmGrad a{};
    a.q.p = p;
    ssm_layout(a.q, plan.scan, ws);
    a.q.state_chunk = 64 / plan.sub;
    char *at = ws + plan.scan.bytes(), *other = at;  // segment states of the walk from the right
    at += plan.scan.state_bytes + plan.scan.log_bytes;
    float *states = reinterpret_cast<float *>(at), *gstates = reinterpret_cast<float *>(at + plan.state_bytes);
    at += 2 * plan.state_bytes;
    if (plan.splits > 1) {
        a.part_B = reinterpret_cast<float *>(at);
        a.part_C = reinterpret_cast<float *>(at + plan.part_bytes);
    }
    a.scalars = reinterpret_cast<float *>(at + 2 * plan.part_bytes);
    a.states = states; a.gstates = gstates;
    a.d_y = o.d_y; a.dx = o.dx; a.ddt = o.ddt; a.dB = o.dB; a.dC = o.dC;
    a.heads_per_block = plan.heads_per_block; a.splits = plan.splits;
    hipError_t e = p.cu_seqlens ? launch_ssm_table(a.q, s) : hipSuccess;
    if (e != hipSuccess) return e;
    // the states entering the chunks from the left ...
    SsmScan f = a.q;
    f.p.final_state = nullptr; f.p.chunk_states = states; f.p.y = nullptr;
    // ... and their gradients from the right: C in B's place, dy in x's
    SsmScan r = a.q;
    r.p.Bm = p.Cm; r.p.b_sb = p.c_sb; r.p.b_st = p.c_st;
    r.p.x = o.d_y; r.p.x_st = static_cast<int64_t>(p.H) * p.P; r.p.x_sb = r.p.x_st * p.T;
    r.p.initial_state = o.d_final; r.p.final_state = o.d_initial; r.p.chunk_states = gstates; r.p.y = nullptr;
    if (plan.scan.split) {
        r.seg_state = reinterpret_cast<float *>(other);
        r.seg_log = reinterpret_cast<float *>(other + plan.scan.state_bytes);
    }
    e = launch_ssm_both(f, r, plan.scan, in_dtype, s);
    if (e != hipSuccess) return e;
    e = in_dtype == 0 ? ssm_grad_f32(a, s) : ssm_grad_bf16(a, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ssm_scalar_kernel, dim3(3 * p.H), dim3(256), 0, s, a, plan.items, plan.sub, o.dA, o.dD, o.ddt_bias);
    return hipGetLastError();
}

}  // namespace kda
