// Latent attention's absorbed form on the fp32 matrix cores, and the join of
// the pieces for both types.
//
// A workgroup takes 16 rows (token, head) and a run of the cache, 32 rows a
// step, staged in LDS as fp32.  S^T = K Q^T: two waves to each 16 keys, half of
// the channels each; the halves meet in LDS, where every wave then reads all of
// S^T and makes the same statistics and probabilities, in the layout that the
// second product wants (register j = key 4 g + j of the lane's row).
// O^T += C^T P^T: each wave a quarter of the latent channels.  One LDS buffer: the
// loop waits for its page lookups and rows.  128 sequences of up to 16384 rows, 32
// heads: 1.84 ms, 1.3 TB/s; 4 of up to 700, 8 heads: 13 us and 7 for the join.
#include "kda_latent_decode.hpp"

namespace kda {

namespace {

constexpr int kRows = kDecodeRowsF32, kKeys = kDecodeKeysF32, kThreads = 256;

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
template <typename O, int DK, int DC>
__global__ void __launch_bounds__(kThreads) decode_f32_kernel(LatentDecodeParams p, int tiles) {
    constexpr int LD = DK + 4, HALF = DK / 2, NB = DC / 64;
    __shared__ float s_k[kKeys * LD];
    __shared__ float s_s[2][kKeys][kRows + 1];
    __shared__ DecodeShared<kThreads> s_run;
    __shared__ const float *s_row[kKeys];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c16 = lane & 15;
    const int tile = blockIdx.x % tiles, worker = blockIdx.x / tiles;
    DecodeRun run = decode_run<kThreads, kKeys>(p, worker, s_run);
    const int d = p.dc + p.dr, rows = p.m * p.H;
    const int row = tile * kRows + c16, t = row / p.H, h = row - t * p.H;  // the lane's row
    const float c = p.scale * kLog2e;
    bool first = true;
    while (run.left > 0) {
        const int n = decode_rows(p, run.b);
        const int64_t steps = (n + kKeys - 1) / kKeys;
        if (steps == 0) { ++run.b; continue; }
        const int64_t s0 = first ? run.at - run.before : 0, count = min(run.left, steps - s0);
        if (s0 == 0 && tile == 0 && tid == 0) p.info[run.b] = decode_info(first, run.per, run.before, steps, worker);
        f32x4 qf[HALF / 16], acc[NB];
        const float *q = static_cast<const float *>(p.q) + run.b * p.q_sb + t * p.q_st + h * p.q_sh;
#pragma unroll
        for (int s = 0; s < HALF / 16; ++s) {
            const int ch = (wave >> 1) * HALF + 16 * s + 4 * g;
            qf[s] = row < rows && ch < d ? load4(q + ch) : f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        float top = -INFINITY, sum = 0.f;
        const int limit = n - p.m + 1 + t;  // keys that the lane's row sees
        for (int64_t i = s0; i < s0 + count; ++i) {
            const int k0 = static_cast<int>(i) * kKeys;
            __syncthreads();
            if (tid < kKeys) {  // the rows' places; rows behind the end stand for row 0 of the step (their weight is 0)
                const int k = k0 + tid < n ? k0 + tid : k0;
                const int page = k / p.page_size;
                int id = p.page_table[run.b * p.table_stride + page];
                const bool bad = id < 0 || id >= p.num_pages;
                if (bad) id = 0;
                if (p.status && (bad || p.lengths[run.b] != n)) *p.status = kBadPages;
                s_row[tid] = static_cast<const float *>(p.cache) + id * p.page_stride + static_cast<int64_t>(k - page * p.page_size) * p.row_stride;
            }
            __syncthreads();
            for (int e = tid; e < kKeys * (DK / 4); e += kThreads) {
                const int r = e / (DK / 4), ch = 4 * (e % (DK / 4));
                *reinterpret_cast<f32x4 *>(s_k + r * LD + ch) = ch < d ? load4(s_row[r] + ch) : f32x4{0.f, 0.f, 0.f, 0.f};
            }
            __syncthreads();
            {
                f32x4 s = {0.f, 0.f, 0.f, 0.f}, odd = s;  // two chains: half as long, for time and for rounding
                const float *at = s_k + ((wave & 1) * 16 + c16) * LD + (wave >> 1) * HALF + 4 * g;
#pragma unroll
                for (int k = 0; k < HALF / 16; ++k) {
                    const f32x4 a = *reinterpret_cast<const f32x4 *>(at + 16 * k);
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        s = mfma_f32(a[j], qf[k][j], s);
                        odd = mfma_f32(a[j + 1], qf[k][j + 1], odd);
                    }
                }
                s += odd;
#pragma unroll
                for (int j = 0; j < 4; ++j) s_s[wave >> 1][(wave & 1) * 16 + 4 * g + j][c16] = s[j];
            }
            __syncthreads();
            float x[8], most = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = 16 * (e >> 2) + 4 * g + (e & 3);
                x[e] = k0 + k < min(n, limit) ? (s_s[0][k][c16] + s_s[1][k][c16]) * c : -INFINITY;
                most = fmaxf(most, x[e]);
            }
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(top, fmaxf(most, __shfl_xor(most, 32)));
            const float base = most == -INFINITY ? 0.f : most;
            const float keep = fast_exp2(top - base);
            top = most;
            sum *= keep;
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[b] *= keep;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = fast_exp2(x[e] - base);
                sum += x[e];
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[b] = mfma_f32(s_k[(16 * (e >> 2) + 4 * g + (e & 3)) * LD + (wave * NB + b) * 16 + c16], x[e], acc[b]);
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        const bool whole = count == steps;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
        if (row < rows) {
            const int64_t slot = static_cast<int64_t>(tile) * 2 * p.workers + 2 * worker + (first ? 0 : 1);
            const int64_t out = static_cast<int64_t>(run.b) * rows + row, part = slot * kRows + c16;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int ch = (wave * NB + b) * 16 + 4 * g;
                if (ch >= p.dc) continue;
                const f32x4 v = acc[b] * inv;
                if (!whole) {
                    *reinterpret_cast<f32x4 *>(p.part_o + part * p.dc + ch) = v;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) io<O>::st(static_cast<O *>(p.o), out * p.dc + ch + j, v[j]);
                }
            }
            if (wave == 0 && g == 0) (whole ? p.lse[out] : p.part_lse[part]) = lse;
        }
        run.left -= count;
        run.at += count;
        run.before += steps;
        ++run.b;
        first = false;
    }
}

// One wave a (sequence, row) whose sequence is in pieces, or empty.
template <typename O>
__global__ void __launch_bounds__(256) join_kernel(LatentDecodeParams p, int tile_rows) {
    const int rows = p.m * p.H;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (id >= static_cast<int64_t>(p.B) * rows) return;
    const int b = static_cast<int>(id / rows), row = static_cast<int>(id - static_cast<int64_t>(b) * rows);
    const int64_t out = id;
    O *o = static_cast<O *>(p.o) + out * p.dc;
    if (decode_rows(p, b) == 0) {
        if (p.status && lane == 0 && row == 0 && p.lengths[b] < 0) *p.status = kBadPages;
        for (int ch = lane; ch < p.dc; ch += 64) io<O>::st(o, ch, 0.f);
        if (lane == 0) p.lse[out] = -INFINITY;
        return;
    }
    const int2 info = p.info[b];
    if (info.y < 0) return;
    const int tile = row / tile_rows;
    const int64_t base = static_cast<int64_t>(tile) * 2 * p.workers, in = row - tile * tile_rows;
    const int w0 = info.x >> 1;
    auto place = [&](int w) { return (base + (w == w0 ? info.x : 2 * w)) * tile_rows + in; };
    float top = -INFINITY;
    for (int w = w0 + lane; w <= info.y; w += 64) top = fmaxf(top, p.part_lse[place(w)]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float ref = top == -INFINITY ? 0.f : top;
    float acc[8], sum = 0.f;  // dc <= 512: lane l holds channels 4 l and 256 + 4 l
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    constexpr int U = 8;  // pieces requested together
    for (int w = w0; w <= info.y; w += U) {
        float lse[U];
        f32x4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = place(min(w + u, info.y));
            lse[u] = w + u <= info.y ? p.part_lse[at] : -INFINITY;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int ch = 256 * e + 4 * lane;
                if (ch < p.dc) v[u][e] = load4(p.part_o + at * p.dc + ch);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (w + u > info.y) break;
            const float wt = fast_exp2((lse[u] - ref) * kLog2e);
            sum += wt;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[4 * e + j] = fmaf(wt, v[u][e][j], acc[4 * e + j]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int ch = 256 * (e >> 2) + 4 * lane + (e & 3);
        if (ch < p.dc) io<O>::st(o, ch, acc[e] * inv);
    }
    if (lane == 0) p.lse[out] = sum == 0.f ? -INFINITY : ref + __builtin_amdgcn_logf(sum) * kLn2;
}

template <typename O>
hipError_t pick_decode(const LatentDecodeParams &p, const LatentDecodePlan &plan, hipStream_t s) {
    const int grid = plan.workers * plan.tiles, d = p.dc + p.dr;
    if (p.dc <= 128 && d <= 192) decode_f32_kernel<O, 192, 128><<<grid, kThreads, 0, s>>>(p, plan.tiles);
    else if (p.dc <= 256 && d <= 320) decode_f32_kernel<O, 320, 256><<<grid, kThreads, 0, s>>>(p, plan.tiles);
    else decode_f32_kernel<O, 576, 512><<<grid, kThreads, 0, s>>>(p, plan.tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_latent_join(const LatentDecodeParams &p, const LatentDecodePlan &plan, int out_dtype, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.B) * p.m * p.H + 3) / 4);
    if (out_dtype == 0) join_kernel<float><<<grid, 256, 0, s>>>(p, plan.rows);
    else join_kernel<bf16_t><<<grid, 256, 0, s>>>(p, plan.rows);
    return hipGetLastError();
}

hipError_t latent_decode_f32(const LatentDecodeParams &p, const LatentDecodePlan &plan, int out_dtype, hipStream_t s) {
    return out_dtype == 0 ? pick_decode<float>(p, plan, s) : pick_decode<bf16_t>(p, plan, s);
}

}  // namespace kda
