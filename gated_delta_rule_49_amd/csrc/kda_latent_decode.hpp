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

// Where a worker's run begins on the line, and how long it is.
struct DecodeRun {
    int64_t left;    // steps of this worker
    int64_t per;     // steps of every worker but the last
    int64_t at;      // the line's step that this worker begins with
    int b;           // the sequence there
    int64_t before;  // the line's steps before that sequence
};
template <int THREADS> struct DecodeShared {
    int64_t wave[THREADS / 64], before;
    int32_t b;
};
// Each thread counts the steps of a run of sequences (one, up to THREADS of them);
// a prefix sum over the threads; the thread with the worker's first step looks for
// it in its own run.
template <int THREADS, int STEP>
__device__ __forceinline__ DecodeRun decode_run(const LatentDecodeParams &p, int worker, DecodeShared<THREADS> &s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int each = (p.B + THREADS - 1) / THREADS, b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
    auto steps = [&](int b) { return (static_cast<int64_t>(decode_rows(p, b)) + STEP - 1) / STEP; };
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) own += steps(b);
    int64_t upto = own;  // with all threads of the wave before
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) s.wave[wave] = upto;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) upto += s.wave[w];
        total += s.wave[w];
    }
    DecodeRun r;
    r.per = (total + p.workers - 1) / p.workers;
    r.at = worker * r.per;
    r.left = min(total, r.at + r.per) - r.at;
    if (r.left > 0 && upto > r.at && upto - own <= r.at) {  // one thread
        int64_t before = upto - own;
        int b = b0;
        for (int64_t n; before + (n = steps(b)) <= r.at; ++b) before += n;
        s.before = before;
        s.b = b;
    }
    __syncthreads();
    r.b = r.left > 0 ? s.b : 0;
    r.before = r.left > 0 ? s.before : 0;
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
