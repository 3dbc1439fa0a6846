// What the absorbed form's kernels share: how the cache's rows are dealt to
// the workgroups, and the join of the pieces.
//
// The rows of all sequences, in steps of STEP rows that never cross a
// sequence's end, form one line; every workgroup takes an equal run of it
// (lengths are only known on the device, and one long sequence beside short
// ones must not leave the card idle).  A run that holds a whole sequence
// writes its result; pieces of a sequence go to the workspace, and the second
// kernel joins them in order.  A run has two pieces at most, its first and its
// last: slots 2 worker and 2 worker + 1.
#pragma once
#include "kda_latent.hpp"

namespace kda {

__device__ __forceinline__ int decode_rows(const LatentDecodeParams &p, int b) {
    const int64_t most = static_cast<int64_t>(p.max_pages) * p.page_size;
    const int n = p.lengths[b];
    return n < 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(n), most));
}

// The line's total steps, and where `worker` begins: sequence, its step there,
// steps to do.  `s_sum` [THREADS / 64]; every thread gets the same values.
struct DecodeRun {
    int64_t left;  // steps of this worker
    int64_t per;   // steps of every worker but the last
    int64_t at;    // the line's step that this worker begins with
    int b;         // the sequence there
    int64_t before;  // the line's steps before that sequence
};
template <int THREADS, int STEP>
__device__ __forceinline__ DecodeRun decode_run(const LatentDecodeParams &p, int worker, int64_t *s_sum) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto steps = [&](int b) -> int64_t { return b < p.B ? (static_cast<int64_t>(decode_rows(p, b)) + STEP - 1) / STEP : 0; };
    int64_t sum = 0;
    for (int b = tid; b < p.B; b += THREADS) sum += steps(b);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < THREADS / 64; ++w) total += s_sum[w];
    DecodeRun r;
    r.per = (total + p.workers - 1) / p.workers;
    r.at = worker * r.per;
    r.left = min(total, r.at + r.per) - r.at;
    r.b = 0;
    r.before = 0;
    if (r.left <= 0) return r;
    for (int b0 = 0; b0 < p.B; b0 += 64) {  // every wave alike: 64 sequences at a time
        const int64_t own = steps(b0 + lane);
        int64_t run = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up(run, d);
            if (lane >= d) run += o;
        }
        const uint64_t past = __ballot(r.before + run > r.at);
        if (past) {
            const int k = __ffsll(static_cast<long long>(past)) - 1;
            r.before += __shfl(run - own, k);
            r.b = b0 + k;
            return r;
        }
        r.before += __shfl(run, 63);
    }
    return r;
}

// Where a sequence's pieces are, from the worker that has its first step, as the
// `first` of its run or not: (first slot, last worker); the workers behind have
// theirs in their first slot.  (0, -1): written whole.
__device__ __forceinline__ int2 decode_info(bool first, int64_t per, int64_t before, int64_t steps, int worker) {
    const int last = static_cast<int>((before + steps - 1) / per);
    return last == worker ? make_int2(0, -1) : make_int2(2 * worker + (first ? 0 : 1), last);
}

// the join, for both types
hipError_t launch_latent_join(const LatentDecodeParams &p, const LatentDecodePlan &plan, int out_dtype, hipStream_t s);
constexpr int kDecodeRowsF32 = 16, kDecodeKeysF32 = 32;  // rows of a tile and keys of a step of fp32 inputs
hipError_t latent_decode_f32(const LatentDecodeParams &p, const LatentDecodePlan &plan, int out_dtype, hipStream_t s);

}  // namespace kda
