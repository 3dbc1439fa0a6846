// The table of packed sequences' tiles for the expanded form of latent
// attention, and the check of the offsets that its kernels read first.
#include "kda_latent.hpp"

namespace kda {

namespace {

// One workgroup.  Each thread takes a run of sequences, the tiles before its
// run come from a prefix sum over the threads.
__device__ __forceinline__ void fill(const int32_t *cu, int total_tokens, int N, int size, int bound, int2 *entry, int32_t *count,
                                     int *s_wave, int *s_bad) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int per = (N + 1023) / 1024;
    const int n0 = min(N, tid * per), n1 = min(N, n0 + per);
    int local = 0;
    for (int n = n0; n < n1; ++n) {
        const int32_t a = cu[n], b = cu[n + 1];
        if (b < a || a < 0 || b > total_tokens) *s_bad = 1;  // any writer sets 1
        else local += (b - a + size - 1) / size;
    }
    if (tid == 0 && (cu[0] != 0 || cu[N] != total_tokens)) *s_bad = 1;
    int run = local;  // inclusive over the threads
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(run, d);
        if (lane >= d) run += o;
    }
    if (lane == 63) s_wave[tid >> 6] = run;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < (tid >> 6)) run += s_wave[w];
        total += s_wave[w];
    }
    // sequences that do not overlap have no more tiles than the bound
    if (total > bound) *s_bad = 1;
    __syncthreads();
    if (*s_bad == 0 && entry) {
        int at = run - local;
        for (int n = n0; n < n1; ++n) {
            const int c = (cu[n + 1] - cu[n] + size - 1) / size;
            for (int i = 0; i < c; ++i) entry[at + i] = make_int2(n, i);
            at += c;
        }
    }
    if (tid == 0 && count) *count = static_cast<int32_t>(total);
    __syncthreads();
}

__global__ void __launch_bounds__(1024) latent_table_kernel(LatentTable t) {
    __shared__ int s_wave[16];
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    fill(t.cu_q, t.T, t.N, t.size_q, t.bound_q, t.entry_q, t.word + 1, s_wave, &s_bad);
    fill(t.cu_k, t.S, t.N, t.size_k, t.bound_k, t.entry_k, t.word + 2, s_wave, &s_bad);
    if (threadIdx.x == 0) {
        const int32_t st = s_bad ? kBadSeqlens : 0;
        t.word[0] = st;
        if (t.user_status) *t.user_status = st;
    }
}

__global__ void status_word_kernel(int32_t *word) { *word = 0; }

}  // namespace

hipError_t launch_latent_table(const LatentTable &t, hipStream_t s) {
    latent_table_kernel<<<1, 1024, 0, s>>>(t);
    return hipGetLastError();
}

hipError_t launch_status_word(int32_t *word, hipStream_t s) {
    status_word_kernel<<<1, 1, 0, s>>>(word);
    return hipGetLastError();
}

}  // namespace kda
