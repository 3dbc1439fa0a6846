// Host side of the state space scan (how it is split, its workspace), the
// tables of packed sequences and the chaining of the segments' states.
#include "kda_ssm_scan.hpp"

namespace kda {

namespace {

// One workgroup: seg_off / chunk_off = first segment / chunk of every
// sequence (an empty sequence has one empty segment, which hands its state
// through), seg_info per segment, and the check of the offsets that every
// later kernel reads first.
__global__ void __launch_bounds__(1024) ssm_table_kernel(SsmScan q, int32_t *seg_off, int4 *seg_info, int32_t *chunk_off,
                                                         int32_t *status) {
    __shared__ int2 s_wave[16];
    __shared__ int32_t s_bad;
    const int tid = threadIdx.x, lane = tid & 63, N = q.p.N;
    const int32_t *cu = q.p.cu_seqlens;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    const int per = (N + 1023) / 1024;
    const int n0 = min(N, tid * per), n1 = min(N, n0 + per);
    auto count = [&](int n) {  // (segments, chunks); a bad length counts as none
        const int len = cu[n + 1] - cu[n];
        const int chunks = len > 0 && len <= q.p.T ? (len + 63) / 64 : 0;
        return make_int2(max(1, (chunks + q.seg_chunks - 1) / q.seg_chunks), chunks);
    };
    int2 local = make_int2(0, 0);
    for (int n = n0; n < n1; ++n) {
        const int32_t a = cu[n], b = cu[n + 1];
        if (b < a || a < 0 || b > q.p.T) s_bad = 1;  // any writer sets 1
        const int2 c = count(n);
        local.x += c.x;
        local.y += c.y;
    }
    if (tid == 0 && (cu[0] != 0 || cu[N] != q.p.T)) s_bad = 1;
    int2 run = local;  // inclusive over the threads
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int ox = __shfl_up(run.x, d), oy = __shfl_up(run.y, d);
        if (lane >= d) { run.x += ox; run.y += oy; }
    }
    if (lane == 63) s_wave[tid >> 6] = run;
    __syncthreads();
    int2 total = make_int2(0, 0);
    for (int w = 0; w < 16; ++w) {
        if (w < (tid >> 6)) { run.x += s_wave[w].x; run.y += s_wave[w].y; }
        total.x += s_wave[w].x;
        total.y += s_wave[w].y;
    }
    // segments beyond the bound only come from bad offsets
    const bool bad = s_bad || total.x > q.segs_bound;
    int at = run.x - local.x, ch = run.y - local.y;
    for (int n = n0; n < n1; ++n) {
        seg_off[n] = at;
        chunk_off[n] = ch;
        const int2 c = count(n);
        if (!bad)
            for (int s = 0; s < c.x; ++s) {
                const int t0 = s * q.seg_chunks * 64;
                seg_info[at + s] = make_int4(cu[n] + t0, min(cu[n + 1] - cu[n] - t0, q.seg_chunks * 64), n, s);
            }
        at += c.x;
        ch += c.y;
    }
    if (tid == 1023) {
        seg_off[N] = total.x;
        chunk_off[N] = total.y;
        *status = bad ? 6 /* KDA_ERR_BAD_SEQLENS */ : 0;
        if (q.user_status) *q.user_status = bad ? 6 : 0;
    }
}

// One thread per 4 state elements of a (sequence, head), walking the
// sequence's segments; four segments' end states are requested together.
__device__ __forceinline__ void combine(const SsmScan &q, const float *first, int block, bool reverse) {
    const int H = q.p.H, per = q.p.Ns * q.p.P;
    const int blocks = (per / 4 + 255) / 256;
    const int e = ((block % blocks) * 256 + threadIdx.x) * 4;
    const int nh = block / blocks, n = nh / H, h = nh % H;
    if (e >= per) return;
    int x0 = n * q.segs_per_seq, count = q.segs_per_seq;
    if (q.p.cu_seqlens) {
        if (*q.status != 0) return;
        x0 = q.seg_off[n];
        count = q.seg_off[n + 1] - x0;
    }
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    if (first) S = *reinterpret_cast<const f32x4 *>(first + static_cast<int64_t>(nh) * per + e);
    const int x = reverse ? x0 + count - 1 : x0, step = reverse ? -1 : 1;
    constexpr int U = 4;
    for (int i = 0; i < count; i += U) {
        f32x4 loc[U];
        float dec[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u + 1 < count) {  // the last one has no end state
                const int64_t xh = static_cast<int64_t>(x + (i + u) * step) * H + h;
                loc[u] = *reinterpret_cast<const f32x4 *>(q.seg_state + xh * per + e);
                dec[u] = fast_exp2(q.seg_log[xh]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < count) {
                const int64_t xh = static_cast<int64_t>(x + (i + u) * step) * H + h;
                *reinterpret_cast<f32x4 *>(q.seg_state + xh * per + e) = S;
                if (i + u + 1 < count) S = dec[u] * S + loc[u];
            }
    }
}
// f from the first segment to the last, and with a grid twice as large r from
// the last to the first
__global__ void __launch_bounds__(256) ssm_combine_kernel(SsmScan f, SsmScan r, int blocks) {
    if (blockIdx.x < blocks) combine(f, f.p.initial_state, blockIdx.x, false);
    else combine(r, r.p.initial_state, blockIdx.x - blocks, true);
}

}  // namespace

SsmPlan ssm_plan(const SsmParams &p, bool packed, int walks) {
    SsmPlan r{};
    r.chunks_per_seq = static_cast<int32_t>((static_cast<int64_t>(p.T) + 63) / 64);
    r.chunks_bound = packed ? static_cast<int64_t>(r.chunks_per_seq) + p.N : static_cast<int64_t>(r.chunks_per_seq) * p.N;
    const int pw = p.P < 32 ? p.P : 32;
    const int items = p.H / p.G * (p.P / pw);  // waves of a group
    r.waves = items > 4 ? 8 : 4;
    r.blocks_per_group = (items + r.waves - 1) / r.waves;
    // Equal sequences: one workgroup for each of the 256 CUs, all of one length
    // (32768 tokens, 64 heads of 64 channels, d_state 128: 138 us for phase 1 and
    // 14 us for the chain, against 150 and 25 with 512 workgroups).  Packed ones
    // end in segments of any length: shorter segments level them (8 sequences of
    // 1 to 7001 tokens, d_state 64: 184 + 83 us with 512, 227 + 99 with 256).  A
    // segment has at least 4 chunks: its state is written and read once, which
    // is the traffic of 2 chunks (d_state 128).
    const int64_t per_seg = static_cast<int64_t>(p.G) * r.blocks_per_group * walks;
    int64_t k = packed ? r.chunks_bound * per_seg / 512 : (r.chunks_bound * per_seg + 255) / 256;
    k = std::max<int64_t>(k, 4);
    k = std::min<int64_t>(k, std::max(1, r.chunks_per_seq));
    r.seg_chunks = static_cast<int32_t>(k);
    r.segs_per_seq = std::max<int32_t>(1, static_cast<int32_t>((r.chunks_per_seq + k - 1) / k));
    r.split = r.segs_per_seq > 1;
    r.segs_bound = static_cast<int32_t>(packed ? (r.chunks_per_seq + k - 1) / k + p.N : static_cast<int64_t>(r.segs_per_seq) * p.N);
    const size_t words = 2 * align_up(sizeof(int32_t) * (static_cast<size_t>(p.N) + 1));
    r.table_bytes = kAlign + (packed ? words + align_up(sizeof(int4) * static_cast<size_t>(r.segs_bound)) : 0);
    if (r.split) {
        r.state_bytes = align_up(sizeof(float) * static_cast<size_t>(r.segs_bound) * p.H * p.Ns * p.P);
        r.log_bytes = align_up(sizeof(float) * static_cast<size_t>(r.segs_bound) * p.H);
    }
    return r;
}

void ssm_layout(SsmScan &q, const SsmPlan &plan, char *ws) {
    q.state_chunk = 64;
    q.seg_chunks = plan.seg_chunks; q.segs_bound = plan.segs_bound;
    q.segs_per_seq = plan.segs_per_seq; q.chunks_per_seq = plan.chunks_per_seq;
    const size_t words = align_up(sizeof(int32_t) * (static_cast<size_t>(q.p.N) + 1));
    q.status = reinterpret_cast<int32_t *>(ws);
    q.seg_off = reinterpret_cast<int32_t *>(ws + kAlign);
    q.chunk_off = reinterpret_cast<int32_t *>(ws + kAlign + words);
    q.seg_info = reinterpret_cast<int4 *>(ws + kAlign + 2 * words);
    q.seg_state = plan.split ? reinterpret_cast<float *>(ws + plan.table_bytes) : nullptr;
    q.seg_log = plan.split ? reinterpret_cast<float *>(ws + plan.table_bytes + plan.state_bytes) : nullptr;
}

hipError_t launch_ssm_table(const SsmScan &q, hipStream_t s) {
    hipLaunchKernelGGL(ssm_table_kernel, dim3(1), dim3(1024), 0, s, q, const_cast<int32_t *>(q.seg_off),
                       const_cast<int4 *>(q.seg_info), const_cast<int32_t *>(q.chunk_off), const_cast<int32_t *>(q.status));
    return hipGetLastError();
}

namespace {
hipError_t launch_combine(const SsmScan &f, const SsmScan &r, int walks, hipStream_t s) {
    const int blocks = (f.p.Ns * f.p.P / 4 + 255) / 256 * f.p.N * f.p.H;
    hipLaunchKernelGGL(ssm_combine_kernel, dim3(static_cast<unsigned>(blocks) * walks), dim3(256), 0, s, f, r, blocks);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_ssm_scan(const SsmScan &q, const SsmPlan &plan, int in_dtype, int out_dtype, hipStream_t s) {
    if (plan.split) {
        hipError_t e = launch_ssm_phase(q, plan, 1, in_dtype, out_dtype, s);
        if (e == hipSuccess) e = launch_combine(q, q, 1, s);
        if (e != hipSuccess) return e;
    }
    return launch_ssm_phase(q, plan, 2, in_dtype, out_dtype, s);
}

hipError_t launch_ssm_both(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int in_dtype, hipStream_t s) {
    if (plan.split) {
        hipError_t e = launch_ssm_states(f, r, plan, 1, in_dtype, s);
        if (e == hipSuccess) e = launch_combine(f, r, 2, s);
        if (e != hipSuccess) return e;
    }
    return launch_ssm_states(f, r, plan, 2, in_dtype, s);
}

}  // namespace kda
