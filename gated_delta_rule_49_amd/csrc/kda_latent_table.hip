// The table of packed sequences' tiles for the expanded form of latent
// attention, and the check of the offsets that its kernels read first.
//
// One workgroup.  Each thread counts the tiles of a run of sequences; a prefix
// sum over the threads gives every sequence's first tile; then a thread takes a
// tile, finds its sequence by bisection, and puts it where its bucket of work
// (tokens of the other side that it sees) begins: the largest first, so that the
// last workgroups of a launch are small ones.  A launch takes a tile's heads one
// after another: the largest first over all heads (8 prompts of 0 to 3001 tokens
// behind 0 to 4097 cached ones, 32 heads, bf16: the forward took 320 us so, head by
// head 348).  The order inside a bucket is that of arrival; no result depends on
// it.  One workgroup's latency bounds it: 8 to 13 us.
#include "kda_latent.hpp"

namespace kda {

namespace {

constexpr int kThreads = 1024, kBuckets = 64;  // buckets: a wave
constexpr int kInLds = 4096;  // sequences whose offsets fit

struct Scratch {
    int off[kInLds + 1];
    int2 len[kInLds];  // of this side, of the other
    int wave[kThreads / 64];
    int bucket[kBuckets + 1];
    int most, bad;
};

// sum over the workgroup of the threads before this one, and of all
__device__ __forceinline__ int2 prefix(int own, int *s_wave) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int run = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(run, d);
        if (lane >= d) run += o;
    }
    if (lane == 63) s_wave[wave] = run;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) before += s_wave[w];
        total += s_wave[w];
    }
    __syncthreads();
    return make_int2(before + run - own, total);
}

// whether cu is 0 = cu[0] <= .. <= cu[N] = tokens (any writer sets bad)
__device__ __forceinline__ void check(const int32_t *cu, int tokens, int N, int *bad) {
    for (int n = threadIdx.x; n < N; n += kThreads) {
        const int32_t a = cu[n], b = cu[n + 1];
        if (b < a || a < 0 || b > tokens) *bad = 1;
    }
    if (threadIdx.x == 0 && (cu[0] != 0 || cu[N] != tokens)) *bad = 1;
}

// work(tokens of this side, of the other, tile) -> tokens of the other side that the tile sees
template <typename W>
__device__ __forceinline__ void fill(const int32_t *cu, const int32_t *other, int N, int size, int bound, int *spill, int2 *entry, int32_t *count, Scratch &s, W &&work) {
    const int tid = threadIdx.x;
    int *off = N <= kInLds ? s.off : spill;  // .. and lengths too in LDS, or read again
    const int per = (N + kThreads - 1) / kThreads;
    const int n0 = min(N, tid * per), n1 = min(N, n0 + per);
    const bool small = N <= kInLds;
    auto length = [&](int n) { return small ? s.len[n] : make_int2(cu[n + 1] - cu[n], other[n + 1] - other[n]); };
    auto tiles = [&](int n) { return (length(n).x + size - 1) / size; };
    int own = 0, most = 0;
    for (int n = n0; n < n1; ++n) {
        if (small) s.len[n] = make_int2(cu[n + 1] - cu[n], other[n + 1] - other[n]);
        own += tiles(n);
        most = max(most, length(n).y);
    }
    if (tid <= kBuckets) s.bucket[tid] = 0;
    if (tid == 0) s.most = 0;
    const int2 at = prefix(own, s.wave);
    atomicMax(&s.most, most);
    int first = at.x;
    for (int n = n0; n < n1; ++n) {
        off[n] = first;
        first += tiles(n);
    }
    if (tid == 0) off[N] = at.y;
    __syncthreads();
    const int total = min(at.y, bound);
    const float scale = static_cast<float>(kBuckets) / static_cast<float>(s.most + 1);
    auto place = [&](int t) {  // (sequence, tile of it, bucket)
        int lo = 0, hi = N;    // the last sequence with off <= t: one with tiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (off[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int i = t - off[lo];
        const int2 len = length(lo);
        const int w = max(0, work(len.x, len.y, i));
        return make_int3(lo, i, kBuckets - 1 - min(kBuckets - 1, static_cast<int>(static_cast<float>(w) * scale)));
    };
    for (int t = tid; t < total; t += kThreads) atomicAdd(&s.bucket[place(t).z + 1], 1);
    __syncthreads();
    if (tid < kBuckets) {  // one wave: where each bucket begins
        int run = s.bucket[tid];
#pragma unroll
        for (int d = 1; d < kBuckets; d <<= 1) {
            const int o = __shfl_up(run, d);
            if (tid >= d) run += o;
        }
        s.bucket[tid] = run;
    }
    __syncthreads();
    for (int t = tid; t < total; t += kThreads) {
        const int3 p = place(t);
        entry[atomicAdd(&s.bucket[p.z], 1)] = make_int2(p.x, p.y);
    }
    if (tid == 0) *count = total;
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads) latent_table_kernel(LatentTable t) {
    __shared__ Scratch s;
    if (threadIdx.x == 0) s.bad = 0;
    __syncthreads();
    check(t.cu_q, t.T, t.N, &s.bad);
    check(t.cu_k, t.S, t.N, &s.bad);
    __syncthreads();
    const bool bad = s.bad != 0;
    if (!bad) {
        const bool causal = t.causal;
        if (t.entry_q)
            fill(t.cu_q, t.cu_k, t.N, t.size_q, t.bound_q, t.spill, t.entry_q, t.word + 1, s,
                 [&](int tq, int tk, int i) { return causal ? min(tk, min(tq, (i + 1) * t.size_q) + tk - tq) : tk; });
        if (t.entry_k)
            fill(t.cu_k, t.cu_q, t.N, t.size_k, t.bound_k, t.spill, t.entry_k, t.word + 2, s,
                 [&](int tk, int tq, int i) { return causal ? tq - max(0, i * t.size_k - (tk - tq)) : tq; });
    }
    if (threadIdx.x == 0) {
        t.word[0] = bad ? kBadSeqlens : 0;
        if (t.user_status) *t.user_status = bad ? kBadSeqlens : 0;
    }
}

__global__ void status_word_kernel(int32_t *word) { *word = 0; }

}  // namespace

size_t latent_table_spill(int N) { return N <= kInLds ? 0 : sizeof(int32_t) * (static_cast<size_t>(N) + 1); }

hipError_t launch_latent_table(const LatentTable &t, hipStream_t s) {
    latent_table_kernel<<<1, kThreads, 0, s>>>(t);
    return hipGetLastError();
}

hipError_t launch_status_word(int32_t *word, hipStream_t s) {
    status_word_kernel<<<1, 1, 0, s>>>(word);
    return hipGetLastError();
}

}  // namespace kda
