// Gradients of latent attention's expanded form: what both types share, and the
// bf16 kernels.  With P = e^(S - lse), dP = dO V^T, delta = rowsum(dO o):
//     dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// A query that sees one key has P = 1 whatever its score: its dS is 0, not what the
// roundings of two equal sums leave of their difference.
//
// Two kernels that each make S and dP again (seven products where one kernel
// would do with five): one owns queries, one owns keys, so that every sum is
// taken in order in one place.  The sums over queries as atomics would save two
// products in seven and change their rounding from run to run.
//
// Queries: as the forward, a wave 32 queries, S^T and dP^T by rows of K and V,
// dQ^T += K^T dS^T by columns of K.
//
// Keys: a workgroup takes 128 keys and walks the queries 64 at a time; 32 keys
// belong to a PAIR of waves, which a SIMD runs side by side.  The first makes S
// and P and keeps dV (K as operand, 64 registers of result), the second makes dP,
// takes P from LDS in fp32 and keeps dK (V as operand, 96 registers).  One wave
// for both would need 300 registers and leave a SIMD no second wave; so the
// exponentials of one run under the products of the other, 40 products each.
//
// P and dS enter their second products as one bf16 operand, which rounds each term
// of a sum by up to 2^-8 of itself, or, where the caller asks for it (precise), as
// two, which round by 2^-16.  Both sides, the call below: 1299 us for 1810; the
// error of bf16 gradients against 64 bits 2.5e-3 for 1.8e-3, what their own
// rounding and that of a bf16 o make.
//
// 2 x 4096 tokens of 32 heads (keys 192, values 128, causal), bf16: queries 575 us
// (three products, 960 TFLOP/s), keys 840 us (four, 820 TFLOP/s), the statistics
// and dk_rope's sum 33 and 13 us (bound by memory), in a short profiled run; a call
// in a long row of them, at a higher clock, takes 1.3 ms in all.  Matrix instructions take 54 %
// and 44 % of the cycles, LDS 28 % and 33 %, without bank conflicts.
#include "kda_latent_bf16.hpp"

namespace kda {

namespace {

// lse log2 e and rowsum(d_o o) of every (head, token), 16 lanes each.  A query
// without a key has +infinity for its lse, by which its probabilities are 0.
template <typename T> __device__ __forceinline__ void load8(float (&x)[8], const T *p) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x4 v = reinterpret_cast<const f32x4 *>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = v[j];
        }
    } else {
        frag8 f;
        f.u = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = bf16_to_f32(f.s[i]);
    }
}
template <typename T, typename O>
__global__ void __launch_bounds__(256) stats_kernel(LatentGradParams g) {
    const int64_t rows = static_cast<int64_t>(g.f.B) * g.f.T;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const int lane = threadIdx.x & 15;
    if (id >= rows * g.f.H) return;
    const int64_t row = id / g.f.H;
    const int h = static_cast<int>(id - row * g.f.H), b = static_cast<int>(row / g.f.T), t = static_cast<int>(row - static_cast<int64_t>(b) * g.f.T);
    float s = 0.f;
    if (8 * lane < g.f.dv) {
        float o[8], d[8];
        load8(o, static_cast<const O *>(g.f.o) + b * g.o_sb + t * g.o_st + h * g.o_sh + 8 * lane);
        load8(d, static_cast<const T *>(g.d_o) + b * g.d_sb + t * g.d_st + h * g.d_sh + 8 * lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(o[i], d[i], s);
    }
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) s += __shfl_xor(s, x);
    if (lane == 0) {
        const float lse = g.f.lse[b * g.l_sb + t * g.l_st + h * g.l_sh];
        g.lse2[h * rows + row] = lse == -INFINITY ? INFINITY : lse * kLog2e;
        g.delta[h * rows + row] = s;
    }
}

// dk_rope: the heads' shares added in order, eight requested together
template <typename T>
__global__ void __launch_bounds__(256) rope_sum_kernel(LatentGradParams g) {
    if (g.f.cu_q && *g.f.status != 0) return;
    const int64_t plane = static_cast<int64_t>(g.f.B) * g.f.S * g.f.dr;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (at >= plane) return;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int h = 0; h < g.f.H; h += 8) {
        f32x4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i < g.f.H) v[i] = *reinterpret_cast<const f32x4 *>(g.dkr_part + (h + i) * plane + at);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i < g.f.H) sum += v[i];
    }
    if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4 *>(static_cast<T *>(g.dkr) + at) = sum;
    else *reinterpret_cast<uint2 *>(static_cast<T *>(g.dkr) + at) = make_uint2(pack2(sum[0], sum[1]), pack2(sum[2], sum[3]));
}

// ------------------------------------------------------------- queries ----
constexpr int kQThreads = 512, kTileQ = kQThreads / 2, kStep = 64;

template <int DK, int DV, int PARTS>
__global__ void __launch_bounds__(kQThreads, 512 / kQThreads) grad_q_bf16_kernel(LatentGradParams gp) {
    constexpr int KB = kStep * DK * 2, VB = kStep * DV * 2;
    __shared__ __attribute__((aligned(128))) char s_tile[2 * (KB + VB)];
    __shared__ uint32_t s_off[kStep * (DK + DV) / 8];  // one a chunk
    const LatentParams &p = gp.f;
    const LatentPlace a = latent_place(p, p.tq, blockIdx.x, p.causal);
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, c32 = lane & 31;
    const bf16_t *kn = static_cast<const bf16_t *>(p.kn) + a.b * p.k_sb + a.h * p.k_sh + a.k0 * p.k_st;
    const bf16_t *kr = static_cast<const bf16_t *>(p.kr) + a.b * p.r_sb + a.k0 * p.r_st;
    const bf16_t *v = static_cast<const bf16_t *>(p.v) + a.b * p.v_sb + a.h * p.v_sh + a.k0 * p.v_st;
    const int q_first = a.tile * kTileQ + wave * 32, qi = q_first + c32;
    const bool inside = qi < a.tq;
    const int shift = a.tk - a.tq;
    const int n = p.causal ? min(a.tk, min(a.tq, (a.tile + 1) * kTileQ) + shift) : a.tk;
    const int n_least = p.causal ? min(n, q_first + shift + 1) : n;
    const int n_wave = q_first >= a.tq ? 0 : p.causal ? min(n, min(a.tq - 1, q_first + 31) + shift + 1) : n;
    const int limit = !inside ? 0 : p.causal ? min(n, qi + shift + 1) : n;

    TileLoader<DK, kStep, kQThreads, BothRead, true, true> keys;
    TileLoader<DV, kStep, kQThreads, BothRead, false, true> values;
    keys.init(kn, p.k_st, p.dn, kr, p.r_st, p.dr, 0, s_off);
    values.init(v, p.v_st, p.dv, v, 0, 0, 0, s_off + kStep * DK / 8);
    const uint32_t lds = lds_address(s_tile);
    if (n > 0) {
        keys.issue(0, n, lds);
        values.issue(0, n, lds + 2 * KB);
    }
    bf16x8 qf[DK / 16], df[DV / 16];
    const int64_t token = static_cast<int64_t>(a.q0) + min(qi, a.tq - 1);
    load_own<DK>(qf, static_cast<const bf16_t *>(p.q) + a.b * p.q_sb + a.h * p.q_sh + token * p.q_st, p.dn + p.dr, kr, 0, inside, h);
    load_own<DV>(df, static_cast<const bf16_t *>(gp.d_o) + a.b * gp.d_sb + a.h * gp.d_sh + token * gp.d_st, p.dv, kr, 0, inside, h);
    const int64_t stat = static_cast<int64_t>(a.h) * p.B * p.T + a.q_row + qi;
    const float lse = inside ? gp.lse2[stat] : 0.f, delta = inside ? gp.delta[stat] : 0.f;
    const float c = p.scale * kLog2e;
    f32x16 acc[DK / 32];
#pragma unroll
    for (int b = 0; b < DK / 32; ++b) acc[b] = zero16();
    const uint32_t key_at = BothRead::row<DK>(lane), value_at = BothRead::row<DV>(lane), column_at = BothRead::columns<DK>(lane);

    for (int k0 = 0, buf = 0; k0 < n; k0 += kStep, buf ^= 1) {
        wait_loads();
        lds_barrier();
        if (k0 + kStep < n) {
            keys.issue(k0 + kStep, n, lds + (buf ^ 1) * KB);
            values.issue(k0 + kStep, n, lds + 2 * KB + (buf ^ 1) * VB);
        }
        if (k0 >= n_wave) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const char *kt = s_tile + buf * KB + 32 * t * DK * 2, *vt = s_tile + 2 * KB + buf * VB + 32 * t * DV * 2;
            f32x16 s = zero16(), dp = zero16();
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                frag8 f;
                f.u = *reinterpret_cast<const uint4 *>(kt + BothRead::step<DK>(key_at, k));
                s = mfma32(f.v, qf[k], s);
            }
#pragma unroll
            for (int k = 0; k < DV / 16; ++k) {
                frag8 f;
                f.u = *reinterpret_cast<const uint4 *>(vt + BothRead::step<DV>(value_at, k));
                dp = mfma32(f.v, df[k], dp);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = fast_exp2(fmaf(s[i], c, -lse));
            if (k0 + kStep > n_least) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3) >= limit) s[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] = s[i] * (dp[i] - delta);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                bf16x8 ds[PARTS];
                half_tile(ds, dp, e);
#pragma unroll
                for (int b = 0; b < DK / 32; ++b) acc[b] = mfma32(BothRead::read_columns<DK>(kt + 16 * e * DK * 2, column_at, b), ds, acc[b]);
            }
        }
    }
    if (!inside) return;
    const float by = limit == 1 ? 0.f : p.scale;
    bf16_t *dq = static_cast<bf16_t *>(gp.dq) + ((a.q_row + qi) * p.H + a.h) * (p.dn + p.dr);
#pragma unroll
    for (int b = 0; b < DK / 32; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (32 * b + 8 * i + 4 * h < p.dn + p.dr) store4(dq + 32 * b + 8 * i + 4 * h, acc[b], i, by);
}

// ---------------------------------------------------------------- keys ----
constexpr int kKThreads = 512, kTileK = 128;

template <int DK, int DV> struct KeyShared {
    float lse[2][kStep], delta[2][kStep];
    f32x4 p[4][2][4][64];  // P of each pair: 32-query tile, four registers, lane
    __attribute__((aligned(128))) char q[2][kStep * DK * 2];
    char d[2][kStep * DV * 2];
};

template <int DK, int DV, int PARTS>
__global__ void __launch_bounds__(kKThreads, 1) grad_k_bf16_kernel(LatentGradParams gp) {
    __shared__ __attribute__((aligned(128))) KeyShared<DK, DV> sh;
    const LatentParams &p = gp.f;
    const LatentPlace a = latent_place(p, gp.tk, blockIdx.x, false);  // early keys are seen by more queries
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), pair = wave & 3;
    const int h = lane >> 5, c32 = lane & 31;
    const int k_first = a.tile * kTileK + pair * 32, ki = k_first + c32;
    const bool inside = ki < a.tk;
    const int64_t token = static_cast<int64_t>(a.k0) + min(ki, a.tk - 1);
    const bf16_t *q = static_cast<const bf16_t *>(p.q) + a.b * p.q_sb + a.h * p.q_sh + a.q0 * p.q_st;
    const bf16_t *d_o = static_cast<const bf16_t *>(gp.d_o) + a.b * gp.d_sb + a.h * gp.d_sh + a.q0 * gp.d_st;
    const int64_t stat = static_cast<int64_t>(a.h) * p.B * p.T + a.q_row;
    const int shift = a.tk - a.tq;
    const float c = p.scale * kLog2e;
    // the first query that sees the tile's first key
    const int start = (p.causal ? max(0, a.tile * kTileK - shift) : 0) / kStep * kStep;

    TileLoader<DK, kStep, kKThreads, BothRead, false> queries;
    TileLoader<DV, kStep, kKThreads, BothRead, false> grads;
    queries.init(q, p.q_st, p.dn + p.dr, q, 0, 0, start);
    grads.init(d_o, gp.d_st, p.dv, d_o, 0, 0, start);
    auto issue = [&](int i0, int buf) {
        queries.issue(i0, a.tq, lds_address(sh.q[0]) + buf * (kStep * DK * 2));
        grads.issue(i0, a.tq, lds_address(sh.d[0]) + buf * (kStep * DV * 2));
        const int64_t at = stat + min(i0 + lane, a.tq - 1);
        if (wave == 0) load_word_to_lds(gp.lse2 + at, lds_address(sh.lse[0]) + buf * (kStep * 4));
        if (wave == 4) load_word_to_lds(gp.delta + at, lds_address(sh.delta[0]) + buf * (kStep * 4));
    };
    if (start < a.tq) issue(start, 0);
    // whether the pair's keys are seen from queries [i0, i0 + 64), and by all of them
    auto seen = [&](int i0) { return !p.causal || i0 + kStep - 1 + shift >= k_first; };
    auto seen_whole = [&](int i0) { return i0 + kStep <= a.tq && (!p.causal || i0 + shift >= k_first + 31); };
    // the query that sees this sequence's first key alone, where the pair has that key
    const int alone = p.causal && k_first == 0 && shift <= 0 ? -shift : -1;
    const uint32_t q_at = BothRead::row<DK>(lane), d_at = BothRead::row<DV>(lane);
    const int64_t key = a.k_row + ki;

    if (wave < 4) {  // S, P, dV
        bf16x8 kf[DK / 16];
        load_own<DK>(kf, static_cast<const bf16_t *>(p.kn) + a.b * p.k_sb + a.h * p.k_sh + token * p.k_st, p.dn,
                     static_cast<const bf16_t *>(p.kr) + a.b * p.r_sb + token * p.r_st, p.dr, inside, h);
        f32x16 acc[DV / 32];
#pragma unroll
        for (int b = 0; b < DV / 32; ++b) acc[b] = zero16();
        const uint32_t column_at = BothRead::columns<DV>(lane);
        for (int i0 = start, buf = 0; i0 < a.tq; i0 += kStep, buf ^= 1) {
            wait_loads();
            lds_barrier();
            if (i0 + kStep < a.tq) issue(i0 + kStep, buf ^ 1);
            const bool work = seen(i0);
            bf16x8 pf[4][PARTS];
            if (work) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x16 s = zero16();
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        frag8 f;
                        f.u = *reinterpret_cast<const uint4 *>(sh.q[buf] + 32 * t * DK * 2 + BothRead::step<DK>(q_at, k));
                        s = mfma32(f.v, kf[k], s);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 lse = *reinterpret_cast<const f32x4 *>(&sh.lse[buf][32 * t + 8 * i + 4 * h]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[4 * i + j] = fast_exp2(fmaf(s[4 * i + j], c, -lse[j]));
                    }
                    if (!seen_whole(i0)) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int qi = i0 + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3);
                            if (qi >= a.tq || (p.causal && ki > qi + shift)) s[i] = 0.f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) sh.p[pair][t][i][lane] = f32x4{s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]};
                    half_tile(pf[2 * t], s, 0);
                    half_tile(pf[2 * t + 1], s, 1);
                }
                const int r = alone - i0;
                if (r >= 0 && r < kStep && h == (r >> 2 & 1)) reinterpret_cast<float *>(&sh.p[pair][r >> 5][(r & 31) >> 3][lane])[r & 3] = 0.f;
            }
            lds_barrier();
            if (work) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int b = 0; b < DV / 32; ++b) acc[b] = mfma32(BothRead::read_columns<DV>(sh.d[buf] + 16 * e * DV * 2, column_at, b), pf[e], acc[b]);
            }
        }
        if (!inside) return;
        bf16_t *dv = static_cast<bf16_t *>(gp.dv) + (key * p.H + a.h) * p.dv;
#pragma unroll
        for (int b = 0; b < DV / 32; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (32 * b + 8 * i + 4 * h < p.dv) store4(dv + 32 * b + 8 * i + 4 * h, acc[b], i, 1.f);
        return;
    }
    // dP, dS, dK
    bf16x8 vf[DV / 16];
    load_own<DV>(vf, static_cast<const bf16_t *>(p.v) + a.b * p.v_sb + a.h * p.v_sh + token * p.v_st, p.dv, q, 0, inside, h);
    f32x16 acc[DK / 32];
#pragma unroll
    for (int b = 0; b < DK / 32; ++b) acc[b] = zero16();
    const uint32_t column_at = BothRead::columns<DK>(lane);
    for (int i0 = start, buf = 0; i0 < a.tq; i0 += kStep, buf ^= 1) {
        wait_loads();
        lds_barrier();
        if (i0 + kStep < a.tq) issue(i0 + kStep, buf ^ 1);
        const bool work = seen(i0);
        f32x16 dp[2];
        if (work) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                dp[t] = zero16();
#pragma unroll
                for (int k = 0; k < DV / 16; ++k) {
                    frag8 f;
                    f.u = *reinterpret_cast<const uint4 *>(sh.d[buf] + 32 * t * DV * 2 + BothRead::step<DV>(d_at, k));
                    dp[t] = mfma32(f.v, vf[k], dp[t]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 delta = *reinterpret_cast<const f32x4 *>(&sh.delta[buf][32 * t + 8 * i + 4 * h]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dp[t][4 * i + j] -= delta[j];
                }
            }
        }
        lds_barrier();
        if (work) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 pr = sh.p[pair][t][i][lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j) dp[t][4 * i + j] *= pr[j];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    bf16x8 ds[PARTS];
                    half_tile(ds, dp[t], e);
#pragma unroll
                    for (int b = 0; b < DK / 32; ++b) acc[b] = mfma32(BothRead::read_columns<DK>(sh.q[buf] + (32 * t + 16 * e) * DK * 2, column_at, b), ds, acc[b]);
                }
            }
        }
    }
    if (!inside) return;
    const float by = a.tk == 1 ? 0.f : p.scale;
    bf16_t *dkn = static_cast<bf16_t *>(gp.dkn) + (key * p.H + a.h) * p.dn;
    float *part = gp.dkr_part + (static_cast<int64_t>(a.h) * p.B * p.S + key) * p.dr;
#pragma unroll
    for (int b = 0; b < DK / 32; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = 32 * b + 8 * i + 4 * h;
            if (ch < p.dn) store4(dkn + ch, acc[b], i, by);
            else if (ch < p.dn + p.dr) store4(part + ch - p.dn, acc[b], i, by);
        }
}

template <int DK, int DV, int PARTS>
hipError_t run(const LatentGradParams &g, hipStream_t s) {
    const LatentParams &p = g.f;
    const int grid_q = p.cu_q ? p.H * p.tq.bound : p.H * p.N * p.tq.per_seq;
    const int grid_k = p.cu_q ? p.H * g.tk.bound : p.H * p.N * g.tk.per_seq;
    if (p.T) grad_q_bf16_kernel<DK, DV, PARTS><<<grid_q, kQThreads, 0, s>>>(g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.S) grad_k_bf16_kernel<DK, DV, PARTS><<<grid_k, kKThreads, 0, s>>>(g);
    return hipGetLastError();
}
template <int PARTS> hipError_t backward_bf16(const LatentGradParams &g, hipStream_t s) {
    const int dk = g.f.dn + g.f.dr;
    if (dk <= 64 && g.f.dv <= 64) return run<64, 64, PARTS>(g, s);
    if (dk <= 128) return run<128, 128, PARTS>(g, s);
    return run<192, 128, PARTS>(g, s);
}
template <typename T> hipError_t backward(const LatentGradParams &g, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(g.f.B) * g.f.T * g.f.H, shared = static_cast<int64_t>(g.f.B) * g.f.S * g.f.dr;
    const unsigned grid = static_cast<unsigned>((rows + 15) / 16);
    if (rows && g.o_dtype == 0) stats_kernel<T, float><<<grid, 256, 0, s>>>(g);
    if (rows && g.o_dtype != 0) stats_kernel<T, bf16_t><<<grid, 256, 0, s>>>(g);
    hipError_t e = hipGetLastError();  // nothing runs on statistics that were not made
    if (e != hipSuccess) return e;
    e = sizeof(T) == 4 ? latent_backward_f32(g, s) : g.f.precise ? backward_bf16<2>(g, s) : backward_bf16<1>(g, s);
    if (e != hipSuccess) return e;
    if (shared) rope_sum_kernel<T><<<static_cast<unsigned>((shared / 4 + 255) / 256), 256, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace

int latent_grad_tile_q(int dtype, int64_t tokens, int H) { return dtype == 0 ? latent_tile_f32(tokens, H) : kTileQ; }
int latent_grad_tile_k(int dtype, int64_t tokens, int H) { return dtype == 0 ? latent_tile_f32(tokens, H) : kTileK; }

hipError_t launch_latent_backward(const LatentGradParams &g, int in_dtype, hipStream_t s) {
    return in_dtype == 0 ? backward<float>(g, s) : backward<bf16_t>(g, s);
}

}  // namespace kda
