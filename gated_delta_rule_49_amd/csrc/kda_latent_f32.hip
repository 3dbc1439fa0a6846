// Latent attention's expanded form on the fp32 matrix cores: forward and
// gradients for fp32 inputs.
//
// Everything is written with the operand that a wave owns along the COLUMNS of
// the products (v_mfma_f32_16x16x4_f32: A is 16 x 4, lane l holds row l % 16,
// k = l / 16; B likewise by columns; C/D: lane l holds column l % 16, rows
// 4 (l / 16) + j).  The forward and the queries' gradient own 16 queries,
//     S^T = K Q^T,   O^T += V^T P^T,   dP^T = V dO^T,   dQ^T += K^T dS^T,
// the keys' gradient 16 keys,
//     S = Q K^T,     dV^T += dO^T P,   dP = dO V^T,     dK^T += Q^T dS.
// A C tile's register j is then row 4 g + j (g = l / 16) of the wave's column,
// which is what the next product's B operand wants when its contraction takes
// rows {4 g + j : g = 0..3} in step j: P and dS go from accumulator to operand
// without leaving their registers, and the shared operand is read from its
// row-major LDS tile by rows (16 bytes, four steps) or by columns (4 bytes).
// Rows of LDS tiles are 4 floats longer than their channels: 8 rows of a
// 16-byte read then fall on 32 different banks.
//
// A query that sees one key has no gradient of its score, exactly.
//
// Softmax: running maximum and sum per query in fp32; a lane sees the query of
// its column and a quarter of the tile's keys.
//
// 600 tokens of 8 heads (keys 192, values 128): 27 us, five dependent steps of 16
// keys a wave; gradients of documents of 0 to 1201 tokens, 2235 in all, 8 heads:
// queries 169 us, keys 195, with matrix instructions in 37 % of the cycles of one
// wave a SIMD.  4096 tokens of 32 heads: 2.4 ms, gradients 8.2 ms, where products
// alone would take 1.1 and 2.9: the larger tiles have one LDS buffer, nothing is in
// flight during their products.
#include "kda_latent.hpp"

namespace kda {

namespace {

constexpr int kTileQ = 64, kTileK = 64;  // four waves of 16
constexpr int kStep = 32;                // tokens of the other side per step

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ void store4(float *p, const f32x4 &v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ void store4(bf16_t *p, const f32x4 &v) {
    const uint32_t a = static_cast<uint32_t>(f32_to_bf16(v[0])) | static_cast<uint32_t>(f32_to_bf16(v[1])) << 16;
    const uint32_t b = static_cast<uint32_t>(f32_to_bf16(v[2])) | static_cast<uint32_t>(f32_to_bf16(v[3])) << 16;
    *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
}

// four channels from `c` of a key: its own part, the shared part, zeros behind
__device__ __forceinline__ f32x4 key4(const LatentParams &p, const float *kn, const float *kr, int64_t token, int c) {
    if (c < p.dn) return load4(kn + token * p.k_st + c);
    if (c < p.dn + p.dr) return load4(kr + token * p.r_st + c - p.dn);
    return f32x4{0.f, 0.f, 0.f, 0.f};
}

// rows [r0, r0 + kStep) of `n` tokens into an LDS tile; zeros outside
template <int D, typename F>
__device__ __forceinline__ void stage(float *tile, int r0, int n, F &&row4) {
    for (int i = threadIdx.x; i < kStep * (D / 4); i += 256) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (r0 + r < n) v = row4(r0 + r, c);
        *reinterpret_cast<f32x4 *>(tile + r * (D + 4) + c) = v;
    }
}

// C tile of 16 rows of an LDS tile (from `row`) by the wave's 16 columns
template <int D>
__device__ __forceinline__ f32x4 by_rows(const float *tile, int row, const f32x4 (&own)[D / 16], int g, int c16) {
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(tile + (row + c16) * (D + 4) + 16 * s + 4 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = mfma_f32(a[j], own[s][j], acc);
    }
    return acc;
}
// acc (channels by the wave's columns) += tile^T w, w a C tile over rows [row, row + 16)
template <int D>
__device__ __forceinline__ void by_cols(f32x4 (&acc)[D / 16], const float *tile, int row, const f32x4 &w, int g, int c16) {
#pragma unroll
    for (int b = 0; b < D / 16; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b] = mfma_f32(tile[(row + 4 * g + j) * (D + 4) + 16 * b + c16], w[j], acc[b]);
}

__device__ __forceinline__ float quarter_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float quarter_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

template <typename O, int DK, int DV>
__global__ void __launch_bounds__(256) prefill_f32_kernel(LatentParams p) {
    __shared__ float s_k[kStep * (DK + 4)], s_v[kStep * (DV + 4)];
    const LatentPlace a = latent_place(p, p.tq, blockIdx.x, p.causal);
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c16 = lane & 15;
    const float *kn = static_cast<const float *>(p.kn) + a.b * p.k_sb + a.h * p.k_sh + a.k0 * p.k_st;
    const float *kr = static_cast<const float *>(p.kr) + a.b * p.r_sb + a.k0 * p.r_st;
    const float *v = static_cast<const float *>(p.v) + a.b * p.v_sb + a.h * p.v_sh + a.k0 * p.v_st;
    const int qi = a.tile * kTileQ + wave * 16 + c16;  // the lane's query
    const float *q = static_cast<const float *>(p.q) + a.b * p.q_sb + a.h * p.q_sh + (static_cast<int64_t>(a.q0) + qi) * p.q_st;
    f32x4 qf[DK / 16];
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        const int c = 16 * s + 4 * g;
        qf[s] = qi < a.tq && c < p.dn + p.dr ? load4(q + c) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int last_q = min(a.tq, (a.tile + 1) * kTileQ) - 1;
    const int shift = a.tk - a.tq;                        // query i sees keys up to i + shift
    const int n = p.causal ? min(a.tk, last_q + shift + 1) : a.tk;
    const int limit = p.causal ? min(n, qi + shift + 1) : n;  // the lane's own
    const float c = p.scale * kLog2e;
    f32x4 acc[DV / 16];
#pragma unroll
    for (int b = 0; b < DV / 16; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    float top = -INFINITY, sum = 0.f;
    for (int k0 = 0; k0 < n; k0 += kStep) {
        __syncthreads();
        stage<DK>(s_k, k0, n, [&](int r, int ch) { return key4(p, kn, kr, r, ch); });
        stage<DV>(s_v, k0, n, [&](int r, int ch) { return ch < p.dv ? load4(v + static_cast<int64_t>(r) * p.v_st + ch) : f32x4{0.f, 0.f, 0.f, 0.f}; });
        __syncthreads();
        f32x4 s[2];
        float most = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = by_rows<DK>(s_k, 16 * t, qf, g, c16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[t][j] = k0 + 16 * t + 4 * g + j < limit ? s[t][j] * c : -INFINITY;
                most = fmaxf(most, s[t][j]);
            }
        }
        most = fmaxf(top, quarter_max(most));
        const float base = most == -INFINITY ? 0.f : most;  // nothing seen yet
        const float keep = fast_exp2(top - base);
        top = most;
        sum *= keep;
#pragma unroll
        for (int b = 0; b < DV / 16; ++b) acc[b] *= keep;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[t][j] = fast_exp2(s[t][j] - base);
                sum += s[t][j];
            }
            by_cols<DV>(acc, s_v, 16 * t, s[t], g, c16);
        }
    }
    sum = quarter_sum(sum);
    if (qi >= a.tq) return;
    const int64_t row = (a.q_row + qi) * p.H + a.h;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    O *o = static_cast<O *>(p.o) + row * p.dv;
#pragma unroll
    for (int b = 0; b < DV / 16; ++b)
        if (16 * b + 4 * g < p.dv) store4(o + 16 * b + 4 * g, acc[b] * inv);
    if (g == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <int DK, int DV>
__global__ void __launch_bounds__(256) grad_q_f32_kernel(LatentGradParams gp) {
    __shared__ float s_k[kStep * (DK + 4)], s_v[kStep * (DV + 4)];
    const LatentParams &p = gp.f;
    const LatentPlace a = latent_place(p, p.tq, blockIdx.x, p.causal);
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c16 = lane & 15;
    const float *kn = static_cast<const float *>(p.kn) + a.b * p.k_sb + a.h * p.k_sh + a.k0 * p.k_st;
    const float *kr = static_cast<const float *>(p.kr) + a.b * p.r_sb + a.k0 * p.r_st;
    const float *v = static_cast<const float *>(p.v) + a.b * p.v_sb + a.h * p.v_sh + a.k0 * p.v_st;
    const int qi = a.tile * kTileQ + wave * 16 + c16;
    const bool inside = qi < a.tq;
    const int64_t row = (a.q_row + qi) * p.H + a.h;
    const float *q = static_cast<const float *>(p.q) + a.b * p.q_sb + a.h * p.q_sh + (static_cast<int64_t>(a.q0) + qi) * p.q_st;
    const float *d_o = static_cast<const float *>(gp.d_o) + a.b * gp.d_sb + a.h * gp.d_sh + (static_cast<int64_t>(a.q0) + qi) * gp.d_st;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 qf[DK / 16], df[DV / 16], acc[DK / 16];
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        const int c = 16 * s + 4 * g;
        qf[s] = inside && c < p.dn + p.dr ? load4(q + c) : zero;
        acc[s] = zero;
    }
#pragma unroll
    for (int s = 0; s < DV / 16; ++s) {
        const int c = 16 * s + 4 * g;
        df[s] = inside && c < p.dv ? load4(d_o + c) : zero;
    }
    const int64_t at = static_cast<int64_t>(a.h) * p.B * p.T + a.q_row + qi;
    const float lse = inside ? gp.lse2[at] : 0.f, delta = inside ? gp.delta[at] : 0.f;
    const int last_q = min(a.tq, (a.tile + 1) * kTileQ) - 1, shift = a.tk - a.tq;
    const int n = p.causal ? min(a.tk, last_q + shift + 1) : a.tk;
    const int limit = inside ? (p.causal ? min(n, qi + shift + 1) : n) : 0;
    const float c = p.scale * kLog2e, by = limit == 1 ? 0.f : p.scale;
    for (int k0 = 0; k0 < n; k0 += kStep) {
        __syncthreads();
        stage<DK>(s_k, k0, n, [&](int r, int ch) { return key4(p, kn, kr, r, ch); });
        stage<DV>(s_v, k0, n, [&](int r, int ch) { return ch < p.dv ? load4(v + static_cast<int64_t>(r) * p.v_st + ch) : f32x4{0.f, 0.f, 0.f, 0.f}; });
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 s = by_rows<DK>(s_k, 16 * t, qf, g, c16);
            f32x4 dp = by_rows<DV>(s_v, 16 * t, df, g, c16);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                dp[j] = k0 + 16 * t + 4 * g + j < limit ? fast_exp2(s[j] * c - lse) * (dp[j] - delta) * by : 0.f;
            by_cols<DK>(acc, s_k, 16 * t, dp, g, c16);
        }
    }
    if (!inside) return;
    float *dq = static_cast<float *>(gp.dq) + row * (p.dn + p.dr);
#pragma unroll
    for (int b = 0; b < DK / 16; ++b)
        if (16 * b + 4 * g < p.dn + p.dr) store4(dq + 16 * b + 4 * g, acc[b]);
}

template <int DK, int DV>
__global__ void __launch_bounds__(256) grad_k_f32_kernel(LatentGradParams gp) {
    __shared__ float s_q[kStep * (DK + 4)], s_d[kStep * (DV + 4)];
    __shared__ float s_lse[kStep], s_delta[kStep];
    const LatentParams &p = gp.f;
    const LatentPlace a = latent_place(p, gp.tk, blockIdx.x, false);  // early keys are seen by more queries
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c16 = lane & 15;
    const int ki = a.tile * kTileK + wave * 16 + c16;  // the lane's key
    const bool inside = ki < a.tk;
    const int64_t token = static_cast<int64_t>(a.k0) + ki;
    const float *kn = static_cast<const float *>(p.kn) + a.b * p.k_sb + a.h * p.k_sh;
    const float *kr = static_cast<const float *>(p.kr) + a.b * p.r_sb;
    const float *v = static_cast<const float *>(p.v) + a.b * p.v_sb + a.h * p.v_sh + token * p.v_st;
    const float *q = static_cast<const float *>(p.q) + a.b * p.q_sb + a.h * p.q_sh + a.q0 * p.q_st;
    const float *d_o = static_cast<const float *>(gp.d_o) + a.b * gp.d_sb + a.h * gp.d_sh + a.q0 * gp.d_st;
    const int64_t row0 = static_cast<int64_t>(a.h) * p.B * p.T + a.q_row;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 kf[DK / 16], vf[DV / 16], dk[DK / 16], dv[DV / 16];
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
        kf[s] = inside ? key4(p, kn, kr, token, 16 * s + 4 * g) : zero;
        dk[s] = zero;
    }
#pragma unroll
    for (int s = 0; s < DV / 16; ++s) {
        vf[s] = inside && 16 * s + 4 * g < p.dv ? load4(v + 16 * s + 4 * g) : zero;
        dv[s] = zero;
    }
    const int shift = a.tk - a.tq;
    const float c = p.scale * kLog2e, by = a.tk == 1 ? 0.f : p.scale;
    // the first query that sees the tile's first key
    int i0 = p.causal ? max(0, a.tile * kTileK - shift) : 0;
    i0 = i0 / kStep * kStep;
    for (; i0 < a.tq; i0 += kStep) {
        __syncthreads();
        stage<DK>(s_q, i0, a.tq, [&](int r, int ch) { return ch < p.dn + p.dr ? load4(q + static_cast<int64_t>(r) * p.q_st + ch) : f32x4{0.f, 0.f, 0.f, 0.f}; });
        stage<DV>(s_d, i0, a.tq, [&](int r, int ch) { return ch < p.dv ? load4(d_o + static_cast<int64_t>(r) * gp.d_st + ch) : f32x4{0.f, 0.f, 0.f, 0.f}; });
        if (threadIdx.x < kStep) {
            const int i = i0 + threadIdx.x;
            s_lse[threadIdx.x] = i < a.tq ? gp.lse2[row0 + i] : 0.f;
            s_delta[threadIdx.x] = i < a.tq ? gp.delta[row0 + i] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f32x4 s = by_rows<DK>(s_q, 16 * t, kf, g, c16);
            f32x4 dp = by_rows<DV>(s_d, 16 * t, vf, g, c16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 16 * t + 4 * g + j, i = i0 + r;
                const bool sees = inside && i < a.tq && (!p.causal || ki <= i + shift);
                s[j] = sees ? fast_exp2(s[j] * c - s_lse[r]) : 0.f;
                dp[j] = sees && (!p.causal || i + shift > 0) ? s[j] * (dp[j] - s_delta[r]) * by : 0.f;
            }
            by_cols<DV>(dv, s_d, 16 * t, s, g, c16);
            by_cols<DK>(dk, s_q, 16 * t, dp, g, c16);
        }
    }
    if (!inside) return;
    const int64_t key = a.k_row + ki;
    float *dkn = static_cast<float *>(gp.dkn) + (key * p.H + a.h) * p.dn;
    float *dvp = static_cast<float *>(gp.dv) + (key * p.H + a.h) * p.dv;
    float *part = gp.dkr_part + (static_cast<int64_t>(a.h) * p.B * p.S + key) * p.dr;
#pragma unroll
    for (int b = 0; b < DK / 16; ++b) {
        const int ch = 16 * b + 4 * g;
        if (ch < p.dn) store4(dkn + ch, dk[b]);
        else if (ch < p.dn + p.dr) store4(part + ch - p.dn, dk[b]);
    }
#pragma unroll
    for (int b = 0; b < DV / 16; ++b)
        if (16 * b + 4 * g < p.dv) store4(dvp + 16 * b + 4 * g, dv[b]);
}

// ------------------------------------------------------- few tiles ----
// The same products where there are too few tiles to fill the card: a workgroup
// takes 16 queries (or keys), its waves in turn 16 tokens of the other side, which
// come from the caches to registers (no LDS, no barrier in the loop);
// the waves' sums meet in LDS at the end, in order.
constexpr int kFewTile = 16, kFewWaves = 8;  // waves of the forward; the gradients' take 400 registers a lane, and are four
// Tokens times heads below which these tiles are taken.  Forward and gradients of
// one sequence, us, these against the larger ones (keys of 192, values of 128):
//     600 tokens x 8 heads 32, 106 : 112, 304     2048 x 16  322, 1131 : 527, 1236
//     2048 x 32 (the limit) 620, 2236 : 620, 2033  4096 x 32  2260, 8460 : 2361, 8159
// and of 64 and 64 channels, 2048 x 16 118, 481 : 166, 525, 2048 x 32 228, 933 : 219, 693.
// One limit for both directions and all widths: where these sizes lie it gives away
// 4 % of a forward (4096 x 32, keys of 192), and what lies between them is not measured.
constexpr int64_t kFewBelow = 65536;

// The key's channels as one: its own part, then the shared one (behind both: the
// first again, whose products meet zeros or are not kept).
struct KeyChannels {
    const float *kn, *kr;
    int64_t k_st, r_st;
    int dn, dr;
    // whole: the key fills its D channels, in parts of whole 16: which part a block
    // of 16 is of is then the same in all lanes
    __device__ __forceinline__ bool whole(int D) const { return dn % 16 == 0 && dn + dr == D; }
    struct Row {
        const float *n, *r;
        int dn;
        __device__ __forceinline__ const float *at(int block) const { return (16 * block < dn ? n : r) + 16 * block; }
    };
    __device__ __forceinline__ Row row(int64_t token, int c) const { return {kn + token * k_st + c, kr + token * r_st + c - dn, dn}; }
    __device__ __forceinline__ const float *at(int64_t token, int c) const {
        return c >= dn && c < dn + dr ? kr + token * r_st + (c - dn) : kn + token * k_st + (c < dn ? c : 0);
    }
};
struct Channels {
    const float *x;
    int64_t st;
    int d;
    __device__ __forceinline__ bool whole(int D) const { return d == D; }
    struct Row {
        const float *x;
        __device__ __forceinline__ const float *at(int block) const { return x + 16 * block; }
    };
    __device__ __forceinline__ Row row(int64_t token, int c) const { return {x + token * st + c}; }
    __device__ __forceinline__ const float *at(int64_t token, int c) const { return x + token * st + (c < d ? c : 0); }
};
// 16 tokens from t0 as operand by rows, and by columns; tokens behind the last (n - 1) repeat it.  With
// BLOCKS the addresses of whole channels are made block by block: fewer instructions (gradients of
// 2235 packed tokens 373 -> 358 us), which in the forward cost registers that it lacks (27 -> 32 us).
template <int D, bool BLOCKS, typename C> __device__ __forceinline__ void rows16(f32x4 (&f)[D / 16], const C &x, int t0, int n, int g, int c16) {
    const int64_t t = min(t0 + c16, n - 1);
    if (BLOCKS && x.whole(D)) {
        const auto row = x.row(t, 4 * g);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) f[s] = load4(row.at(s));
        return;
    }
#pragma unroll
    for (int s = 0; s < D / 16; ++s) f[s] = load4(x.at(t, 16 * s + 4 * g));
}
template <int D, bool BLOCKS, typename C> __device__ __forceinline__ void cols16(f32x4 (&f)[D / 16], const C &x, int t0, int n, int g, int c16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t t = min(t0 + 4 * g + j, n - 1);
        if (BLOCKS && x.whole(D)) {
            const auto row = x.row(t, c16);
#pragma unroll
            for (int b = 0; b < D / 16; ++b) f[b][j] = *row.at(b);
        } else {
#pragma unroll
            for (int b = 0; b < D / 16; ++b) f[b][j] = *x.at(t, 16 * b + c16);
        }
    }
}
// two chains: the products of one wait for each other
template <int D> __device__ __forceinline__ f32x4 dot16(const f32x4 (&a)[D / 16], const f32x4 (&own)[D / 16]) {
    f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            x = mfma_f32(a[s][j], own[s][j], x);
            y = mfma_f32(a[s][j + 1], own[s][j + 1], y);
        }
    return x + y;
}
template <int D> __device__ __forceinline__ void add16(f32x4 (&acc)[D / 16], const f32x4 (&cols)[D / 16], const f32x4 &w) {
#pragma unroll
    for (int b = 0; b < D / 16; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b] = mfma_f32(cols[b][j], w[j], acc[b]);
}
// the wave's own 16 tokens; zeros outside
template <int D, typename C> __device__ __forceinline__ void own16(f32x4 (&f)[D / 16], const C &x, int64_t t, int d, bool inside, int g) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const int c = 16 * s + 4 * g;
        f[s] = load4(x.at(t, c));
        if (!inside || c >= d) f[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
}
template <int D> __device__ __forceinline__ void put16(float *to, const f32x4 (&acc)[D / 16], int wave, int g, int c16) {
#pragma unroll
    for (int b = 0; b < D / 16; ++b) *reinterpret_cast<f32x4 *>(to + (wave * 16 + c16) * (D + 4) + 16 * b + 4 * g) = acc[b];
}

struct FewPlace {
    LatentPlace a;
    KeyChannels keys;
    Channels values, queries;
};
__device__ __forceinline__ FewPlace few_place(const LatentParams &p, const LatentTiles &t, bool down) {
    FewPlace f;
    f.a = latent_place(p, t, blockIdx.x, down);
    if (!f.a.valid) return f;
    const LatentPlace &a = f.a;
    f.keys = {static_cast<const float *>(p.kn) + a.b * p.k_sb + a.h * p.k_sh + a.k0 * p.k_st, static_cast<const float *>(p.kr) + a.b * p.r_sb + a.k0 * p.r_st,
              p.k_st, p.r_st, p.dn, p.dr};
    f.values = {static_cast<const float *>(p.v) + a.b * p.v_sb + a.h * p.v_sh + a.k0 * p.v_st, p.v_st, p.dv};
    f.queries = {static_cast<const float *>(p.q) + a.b * p.q_sb + a.h * p.q_sh + a.q0 * p.q_st, p.q_st, p.dn + p.dr};
    return f;
}

template <typename O, int DK, int DV>
__global__ void __launch_bounds__(64 * kFewWaves, 1) prefill_few_kernel(LatentParams p) {
    __shared__ float s_acc[kFewWaves * 16 * (DV + 4)], s_top[kFewWaves][16], s_sum[kFewWaves][16];
    const FewPlace f = few_place(p, p.tq, p.causal);
    const LatentPlace &a = f.a;
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c16 = lane & 15;
    const int q0 = a.tile * kFewTile, qi = q0 + c16, shift = a.tk - a.tq;
    f32x4 qf[DK / 16], acc[DV / 16];
    own16<DK>(qf, f.queries, min(qi, a.tq - 1), p.dn + p.dr, qi < a.tq, g);
#pragma unroll
    for (int b = 0; b < DV / 16; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int n = p.causal ? min(a.tk, min(a.tq, q0 + kFewTile) + shift) : a.tk;
    const int limit = p.causal ? min(n, qi + shift + 1) : n;
    const float c = p.scale * kLog2e;
    float top = -INFINITY, sum = 0.f;
    f32x4 kf[DK / 16];
    if (n > 0) rows16<DK, false>(kf, f.keys, wave * 16, n, g, c16);
    for (int k0 = wave * 16; k0 < n; k0 += 16 * kFewWaves) {
        f32x4 vf[DV / 16];
        cols16<DV, false>(vf, f.values, k0, n, g, c16);
        f32x4 s = dot16<DK>(kf, qf);
        rows16<DK, false>(kf, f.keys, k0 + 16 * kFewWaves, n, g, c16);  // the next step's, under this one's second half
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = k0 + 4 * g + j < limit ? s[j] * c : -INFINITY;
            most = fmaxf(most, s[j]);
        }
        most = fmaxf(top, quarter_max(most));
        const float base = most == -INFINITY ? 0.f : most, keep = fast_exp2(top - base);
        top = most;
        sum *= keep;
#pragma unroll
        for (int b = 0; b < DV / 16; ++b) acc[b] *= keep;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = fast_exp2(s[j] - base);
            sum += s[j];
        }
        add16<DV>(acc, vf, s);
    }
    sum = quarter_sum(sum);
    put16<DV>(s_acc, acc, wave, g, c16);
    if (g == 0) {
        s_top[wave][c16] = top;
        s_sum[wave][c16] = sum;
    }
    __syncthreads();
    constexpr int PARTS = 4 * kFewWaves;
    const int i = threadIdx.x / PARTS, part = threadIdx.x % PARTS;  // a query, four channels of every 4 PARTS
    if (q0 + i >= a.tq) return;
    top = s_top[0][i];
#pragma unroll
    for (int k = 1; k < kFewWaves; ++k) top = fmaxf(top, s_top[k][i]);
    const float base = top == -INFINITY ? 0.f : top;
    float w[kFewWaves];
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) {
        w[k] = fast_exp2(s_top[k][i] - base);
        sum += w[k] * s_sum[k][i];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = (a.q_row + q0 + i) * p.H + a.h;
    O *o = static_cast<O *>(p.o) + row * p.dv;
    for (int ch = 4 * part; ch < p.dv; ch += 4 * PARTS) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kFewWaves; ++k) v += w[k] * load4(s_acc + (k * 16 + i) * (DV + 4) + ch);
        store4(o + ch, v * inv);
    }
    if (part == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <int DK, int DV>
__global__ void __launch_bounds__(256, 1) grad_q_few_kernel(LatentGradParams gp) {
    __shared__ float s_acc[4 * 16 * (DK + 4)];
    const LatentParams &p = gp.f;
    const FewPlace f = few_place(p, p.tq, p.causal);
    const LatentPlace &a = f.a;
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c16 = lane & 15;
    const int q0 = a.tile * kFewTile, qi = q0 + c16, shift = a.tk - a.tq;
    const bool inside = qi < a.tq;
    const Channels grads = {static_cast<const float *>(gp.d_o) + a.b * gp.d_sb + a.h * gp.d_sh + a.q0 * gp.d_st, gp.d_st, p.dv};
    f32x4 qf[DK / 16], df[DV / 16], acc[DK / 16];
    own16<DK>(qf, f.queries, min(qi, a.tq - 1), p.dn + p.dr, inside, g);
    own16<DV>(df, grads, min(qi, a.tq - 1), p.dv, inside, g);
#pragma unroll
    for (int b = 0; b < DK / 16; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t at = static_cast<int64_t>(a.h) * p.B * p.T + a.q_row + qi;
    const float lse = inside ? gp.lse2[at] : 0.f, delta = inside ? gp.delta[at] : 0.f;
    const int n = p.causal ? min(a.tk, min(a.tq, q0 + kFewTile) + shift) : a.tk;
    const int limit = inside ? (p.causal ? min(n, qi + shift + 1) : n) : 0;
    const float c = p.scale * kLog2e, by = limit == 1 ? 0.f : p.scale;
    f32x4 kf[DK / 16], vf[DV / 16];
    if (n > 0) {
        rows16<DK, true>(kf, f.keys, wave * 16, n, g, c16);
        rows16<DV, true>(vf, f.values, wave * 16, n, g, c16);
    }
    for (int k0 = wave * 16; k0 < n; k0 += 64) {
        f32x4 kc[DK / 16];
        cols16<DK, true>(kc, f.keys, k0, n, g, c16);
        const f32x4 s = dot16<DK>(kf, qf);
        f32x4 dp = dot16<DV>(vf, df);
        rows16<DK, true>(kf, f.keys, k0 + 64, n, g, c16);  // the next step's, under this one's second half
        rows16<DV, true>(vf, f.values, k0 + 64, n, g, c16);
#pragma unroll
        for (int j = 0; j < 4; ++j) dp[j] = k0 + 4 * g + j < limit ? fast_exp2(s[j] * c - lse) * (dp[j] - delta) * by : 0.f;
        add16<DK>(acc, kc, dp);
    }
    put16<DK>(s_acc, acc, wave, g, c16);
    __syncthreads();
    const int i = threadIdx.x >> 4, part = threadIdx.x & 15;
    if (q0 + i >= a.tq) return;
    float *dq = static_cast<float *>(gp.dq) + ((a.q_row + q0 + i) * p.H + a.h) * (p.dn + p.dr);
    for (int ch = 4 * part; ch < p.dn + p.dr; ch += 64) {
        f32x4 v = load4(s_acc + i * (DK + 4) + ch);
#pragma unroll
        for (int k = 1; k < 4; ++k) v += load4(s_acc + (k * 16 + i) * (DK + 4) + ch);
        store4(dq + ch, v);
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(256, 1) grad_k_few_kernel(LatentGradParams gp) {
    __shared__ float s_k[4 * 16 * (DK + 4)], s_v[4 * 16 * (DV + 4)];
    const LatentParams &p = gp.f;
    const FewPlace f = few_place(p, gp.tk, false);
    const LatentPlace &a = f.a;
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c16 = lane & 15;
    const int k0 = a.tile * kFewTile, ki = k0 + c16, shift = a.tk - a.tq;
    const bool inside = ki < a.tk;
    const Channels grads = {static_cast<const float *>(gp.d_o) + a.b * gp.d_sb + a.h * gp.d_sh + a.q0 * gp.d_st, gp.d_st, p.dv};
    f32x4 kf[DK / 16], vf[DV / 16], dk[DK / 16], dv[DV / 16];
    own16<DK>(kf, f.keys, min(ki, a.tk - 1), p.dn + p.dr, inside, g);
    own16<DV>(vf, f.values, min(ki, a.tk - 1), p.dv, inside, g);
#pragma unroll
    for (int b = 0; b < DK / 16; ++b) dk[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < DV / 16; ++b) dv[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t row0 = static_cast<int64_t>(a.h) * p.B * p.T + a.q_row;
    const float c = p.scale * kLog2e, by = a.tk == 1 ? 0.f : p.scale;
    // the first query that sees the tile's first key
    const int start = (p.causal ? max(0, k0 - shift) : 0) / 16 * 16;
    f32x4 qf[DK / 16], df[DV / 16];
    if (a.tq > 0) {
        rows16<DK, true>(qf, f.queries, start + wave * 16, a.tq, g, c16);
        rows16<DV, true>(df, grads, start + wave * 16, a.tq, g, c16);
    }
    for (int i0 = start + wave * 16; i0 < a.tq; i0 += 64) {
        f32x4 qc[DK / 16], dc[DV / 16], lse, delta;
        cols16<DV, true>(dc, grads, i0, a.tq, g, c16);
        cols16<DK, true>(qc, f.queries, i0, a.tq, g, c16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = row0 + min(i0 + 4 * g + j, a.tq - 1);
            lse[j] = gp.lse2[i];
            delta[j] = gp.delta[i];
        }
        f32x4 s = dot16<DK>(qf, kf);
        f32x4 dp = dot16<DV>(df, vf);
        rows16<DK, true>(qf, f.queries, i0 + 64, a.tq, g, c16);  // the next step's, under this one's second half
        rows16<DV, true>(df, grads, i0 + 64, a.tq, g, c16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + 4 * g + j;
            const bool sees = inside && i < a.tq && (!p.causal || ki <= i + shift);
            s[j] = sees ? fast_exp2(s[j] * c - lse[j]) : 0.f;
            dp[j] = sees && (!p.causal || i + shift > 0) ? s[j] * (dp[j] - delta[j]) * by : 0.f;
        }
        add16<DV>(dv, dc, s);
        add16<DK>(dk, qc, dp);
    }
    put16<DK>(s_k, dk, wave, g, c16);
    put16<DV>(s_v, dv, wave, g, c16);
    __syncthreads();
    const int i = threadIdx.x >> 4, part = threadIdx.x & 15;
    if (k0 + i >= a.tk) return;
    const int64_t key = a.k_row + k0 + i;
    float *dkn = static_cast<float *>(gp.dkn) + (key * p.H + a.h) * p.dn, *dvp = static_cast<float *>(gp.dv) + (key * p.H + a.h) * p.dv;
    float *shared = gp.dkr_part + (static_cast<int64_t>(a.h) * p.B * p.S + key) * p.dr;
    for (int ch = 4 * part; ch < p.dn + p.dr; ch += 64) {
        f32x4 v = load4(s_k + i * (DK + 4) + ch);
#pragma unroll
        for (int k = 1; k < 4; ++k) v += load4(s_k + (k * 16 + i) * (DK + 4) + ch);
        store4(ch < p.dn ? dkn + ch : shared + ch - p.dn, v);
    }
    for (int ch = 4 * part; ch < p.dv; ch += 64) {
        f32x4 v = load4(s_v + i * (DV + 4) + ch);
#pragma unroll
        for (int k = 1; k < 4; ++k) v += load4(s_v + (k * 16 + i) * (DV + 4) + ch);
        store4(dvp + ch, v);
    }
}

template <typename O, int DK, int DV>
hipError_t run_prefill(const LatentParams &p, hipStream_t s) {
    const int grid = p.cu_q ? p.H * p.tq.bound : p.H * p.N * p.tq.per_seq;
    if (p.tq.size == kFewTile) prefill_few_kernel<O, DK, DV><<<grid, 64 * kFewWaves, 0, s>>>(p);
    else prefill_f32_kernel<O, DK, DV><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}
template <typename O>
hipError_t pick_prefill(const LatentParams &p, hipStream_t s) {
    const int dk = p.dn + p.dr;
    if (dk <= 64 && p.dv <= 64) return run_prefill<O, 64, 64>(p, s);
    if (dk <= 128) return run_prefill<O, 128, 128>(p, s);
    return run_prefill<O, 192, 128>(p, s);
}

template <int DK, int DV>
hipError_t run_grad(const LatentGradParams &g, hipStream_t s) {
    const LatentParams &p = g.f;
    const int grid_q = p.cu_q ? p.H * p.tq.bound : p.H * p.N * p.tq.per_seq;
    const int grid_k = p.cu_q ? p.H * g.tk.bound : p.H * p.N * g.tk.per_seq;
    if (p.T && p.tq.size == kFewTile) grad_q_few_kernel<DK, DV><<<grid_q, 256, 0, s>>>(g);
    if (p.T && p.tq.size != kFewTile) grad_q_f32_kernel<DK, DV><<<grid_q, 256, 0, s>>>(g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.S && g.tk.size == kFewTile) grad_k_few_kernel<DK, DV><<<grid_k, 256, 0, s>>>(g);
    if (p.S && g.tk.size != kFewTile) grad_k_f32_kernel<DK, DV><<<grid_k, 256, 0, s>>>(g);
    return hipGetLastError();
}
hipError_t pick_grad(const LatentGradParams &g, hipStream_t s) {
    const int dk = g.f.dn + g.f.dr;
    if (dk <= 64 && g.f.dv <= 64) return run_grad<64, 64>(g, s);
    if (dk <= 128) return run_grad<128, 128>(g, s);
    return run_grad<192, 128>(g, s);
}

}  // namespace

int latent_tile_f32(int64_t tokens, int H) { return tokens * H < kFewBelow ? kFewTile : kTileQ; }

hipError_t latent_prefill_f32(const LatentParams &p, int out_dtype, hipStream_t s) {
    return out_dtype == 0 ? pick_prefill<float>(p, s) : pick_prefill<bf16_t>(p, s);
}
hipError_t latent_backward_f32(const LatentGradParams &g, hipStream_t s) { return pick_grad(g, s); }

}  // namespace kda
