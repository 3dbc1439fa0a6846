// Gradients of the selective state space scan, from the state entering every
// chunk (a forward pass over the states alone) and the state gradient arriving
// at every chunk's end (the same pass in reverse over C and dy).  Within a
// chunk, with suf, cum, tot as in kda_ssm_scan.hpp, S = S_in, G = the gradient
// of the state at the chunk's end, and for s <= t
//     D_ts = 2^(suf_s - suf_t),  Q_ts = dy_t . x_s,  K_ts = C_t . B_s,
//     E_ts = Q_ts K_ts D_ts :
//   dC_t = sum_s Q_ts D_ts dt_s B_s + 2^cum_t S dy_t
//   dB_s = sum_t Q_ts D_ts dt_s C_t + dt_s 2^suf_s G x_s
//   du_s = sum_t K_ts D_ts dy_t     + 2^suf_s G^T B_s ,   dx_s = dt_s du_s + D dy_s
//   ddt_s = sum_t E_ts + 2^suf_s B_s . G x_s  +  A dlog_s
//   dlog_t = sum_{i >= t > j} E_ij dt_j + sum_{i >= t} 2^cum_i C_i . S dy_i
//            + sum_{j < t} dt_j 2^suf_j B_j . G x_j + 2^tot <G, S>
// Every exponent is <= 0 for decays, and dlog is a sum over what passes
// through token t, so nothing is recovered as a small difference of sums over
// the sequence.  (The first sum runs over row minus column sums of the same
// E without its diagonal, inside the chunk.)
//
// One workgroup takes a chunk, a group and some of its heads, one after the
// other; wave w owns 16 rows n of the states and the same 16 columns of dB and
// dC, whose sums over the heads stay in its accumulators.  Each head's states
// are read once, straight into operand order.
//
// 2 x 4096 tokens, 32 heads of 64 channels, one group, d_state 128, bf16: 208 us,
// after 2 x 66 us for the states from both ends (each direction by itself took
// 2 x 40) and 11 for their chains, and before 13 for the sums.  One workgroup fits a CU (145184 bytes of LDS); vector
// instructions take 32 % of the cycles, LDS 31 % (14 % conflicts), matrix
// instructions 11 %: it waits at the three barriers of a head.  Rows 16 banks
// apart for what is only read by columns cost more in the writes than they
// gained (4 % slower).  Other shapes are less well served: with 128 bf16 channels
// 30 to 40 registers spill, and fp32 instances keep an operand of the du tiles in
// 64 bytes of scratch a lane.
#pragma once
#include "kda_ssm_scan.hpp"

namespace kda {

namespace {

// the value of lane ^ BIT of the same 16
template <int BIT>
__device__ __forceinline__ float lane_xor(float v) {
    const int x = __builtin_bit_cast(int, v);
    if constexpr (BIT == 1) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, x, 0xb1, 0xf, 0xf, true));       // quad_perm 1,0,3,2
    else if constexpr (BIT == 2) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, x, 0x4e, 0xf, 0xf, true));  // quad_perm 2,3,0,1
    else if constexpr (BIT == 8) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, x, 0x128, 0xf, 0xf, true)); // row_ror:8
    else return __shfl_xor(v, BIT);
}
template <int BIT>
__device__ __forceinline__ double lane_xor(double v) {
    const int2 x = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, make_int2(__builtin_bit_cast(int, lane_xor<BIT>(__builtin_bit_cast(float, x.x))),
                                                __builtin_bit_cast(int, lane_xor<BIT>(__builtin_bit_cast(float, x.y)))));
}
// Sums of V = 4, 8 or 16 values over the 16 lanes of a lane group: each
// exchange halves the values a lane carries; lane c ends with the sum of value
// c / (16 / V).
template <int V, int BIT, typename T>
__device__ __forceinline__ T sum16(const T *v, int c16) {
    if constexpr (V > 1) {
        const bool up = c16 & BIT;
        T next[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) next[i] = (up ? v[i + V / 2] : v[i]) + lane_xor<BIT>(up ? v[i] : v[i + V / 2]);
        return sum16<V / 2, BIT / 2>(next, c16);
    } else if constexpr (BIT > 0) {
        const T next = v[0] + lane_xor<BIT>(v[0]);
        return sum16<1, BIT / 2>(&next, c16);
    } else {
        return v[0];
    }
}

template <typename TI, int NS, int P>
struct GradCfg {
    static constexpr bool BF = std::is_same<TI, bf16_t>::value;
    static constexpr int EX = quad<TI>::PARTS, ORD = BF ? 2 : 3;
    // M1, M2 and, for du, G: they make dx, dB and dC alone, which are rounded to
    // bf16 where the inputs are; two rounded parts are off by 2^-16
    static constexpr int XP = BF ? 2 : 3;
    // the states' products also make the fp32 sums dA and ddt_bias: all three parts
    static constexpr int SP = 3;
    static constexpr int L = BF ? 64 : 32, SUB = 64 / L, ST = L / 16, TK = L / 32;
    static constexpr int NT = NS / 16, NKS = (NS + 31) / 32, PT = P / 16, PKS = (P + 31) / 32;
    static constexpr int RN = NKS * 32 + 8, RP = PKS * 32 + 8, RL = L + 8;
    // LDS, in bf16 elements
    static constexpr int BN = 0, CN = BN + EX * L * RN, XN = CN + EX * L * RN, YN = XN + EX * L * RP;
    static constexpr int M1 = YN + EX * L * RP, M2 = M1 + XP * L * RL, GN = M2 + XP * L * RL;
    // then floats: dt, suf, 2^cum, 2^suf, diagonals of Q and E, suf's rounding; row and column sums per tile (64 bits); inter and outer per wave; <G, S> per wave
    static constexpr int FDT = 0, FSUF = L, FCUM = 2 * L, FWS = 3 * L, FQD = 4 * L, FED = 5 * L, FLO = 6 * L, FR = 7 * L, FC = FR + 2 * ST * L,
                         FI = FC + 2 * ST * L, FO = FI + NT * L, FX = FO + NT * L, FEND = FX + 8;
    // G by rows, for du: through LDS where it fits, else read a second time
    static constexpr bool GLDS = sizeof(bf16_t) * (GN + XP * NS * RP) + sizeof(float) * FEND <= 160 * 1024;
    static constexpr int END = GN + (GLDS ? XP * NS * RP : 0);
    static_assert(END % 4 == 0 && FR % 2 == 0, "64-bit sums are aligned");
    static constexpr size_t BYTES = sizeof(bf16_t) * END + sizeof(float) * FEND;
};

template <typename TI, int NS, int P>
__global__ void __launch_bounds__(512) ssm_grad_kernel(SsmGrad a) {
    using Cf = GradCfg<TI, NS, P>;
    constexpr int EX = Cf::EX, ORD = Cf::ORD, XP = Cf::XP, SP = Cf::SP, L = Cf::L, SUB = Cf::SUB, ST = Cf::ST, TK = Cf::TK, NT = Cf::NT;
    constexpr int NKS = Cf::NKS, PT = Cf::PT, PKS = Cf::PKS, RN = Cf::RN, RP = Cf::RP, RL = Cf::RL;
    __shared__ __attribute__((aligned(16))) char smem[Cf::BYTES];
    bf16_t *lds = reinterpret_cast<bf16_t *>(smem);
    float *fl = reinterpret_cast<float *>(smem + sizeof(bf16_t) * Cf::END);
    double *rsum = reinterpret_cast<double *>(fl + Cf::FR), *csum = reinterpret_cast<double *>(fl + Cf::FC);
    const SsmParams &p = a.q.p;
    int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, g = lane >> 4, c16 = lane & 15;

    // block -> (chunk of 64, part of it, group, split of the group's heads)
    const int block = xcd_order(blockIdx.x, gridDim.x);
    const int per_item = p.G * a.splits;
    const int item = block / per_item, grp = block / a.splits % p.G, split = block % a.splits;
    const int chunk = item / SUB, sub = item % SUB;
    int row, t0, len, items;
    if (p.cu_seqlens) {
        if (*a.q.status != 0 || chunk >= a.q.chunk_off[p.N]) return;
        const int n = chunk_to_seq(a.q.chunk_off, p.N, chunk);
        row = 0;
        t0 = (chunk - a.q.chunk_off[n]) * 64 + sub * L;
        len = min(p.cu_seqlens[n + 1] - p.cu_seqlens[n] - t0, L);
        t0 += p.cu_seqlens[n];
        items = (a.q.chunks_per_seq + p.N) * SUB;
    } else {
        if (chunk >= p.N * a.q.chunks_per_seq) return;
        row = chunk / a.q.chunks_per_seq;
        t0 = (chunk % a.q.chunks_per_seq) * 64 + sub * L;
        len = min(p.T - t0, L);
        items = p.N * a.q.chunks_per_seq * SUB;
    }
    const int hpg = p.H / p.G;
    const int h0 = grp * hpg + split * a.heads_per_block, h1 = min(h0 + a.heads_per_block, (grp + 1) * hpg);
    if (len <= 0) {  // the second part of a short chunk: its share of the sums is zero
        for (int h = h0; h < h1; ++h)
            if (tid < 3) a.scalars[(static_cast<int64_t>(tid) * p.H + h) * items + item] = 0.f;
        return;
    }
    const int64_t flat0 = static_cast<int64_t>(row) * p.T + t0;
    const TI *xb = static_cast<const TI *>(p.x) + row * p.x_sb + t0 * p.x_st;
    const TI *bb = static_cast<const TI *>(p.Bm) + row * p.b_sb + t0 * p.b_st + static_cast<int64_t>(grp) * NS;
    const TI *cb = static_cast<const TI *>(p.Cm) + row * p.c_sb + t0 * p.c_st + static_cast<int64_t>(grp) * NS;

    // A [tokens, width] tile goes into LDS in granule order, 4 tokens by 4
    // columns a thread.  Rows past the chunk are zeros: a token there has step
    // size 0, but it must not meet another's finite factor with what it holds.
    auto load_quad = [&](quad<TI> &v, const TI *src, int64_t stride, int tq, int cq) {
        const uint32_t st = static_cast<uint32_t>(stride);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v.zero(r);
            if (len == L || tq * 4 + r < len) v.ld(r, src + (static_cast<uint32_t>(tq * 4 + r) * st + 4 * cq));
        }
    };
    auto store_quad = [&](const quad<TI> &v, int at, int stride, int tq, int cq) {
#pragma unroll
        for (int part = 0; part < EX; ++part)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<uint2 *>(lds + at + part * L * stride + (tq * 4 + r) * stride + col_pos(cq * 4)) = v.row(r, part).u;
    };
    auto stage = [&](int at, int stride, const TI *src, int64_t st) {
        for (int i = tid; i < (L / 4) * (NS / 4); i += 512) {
            quad<TI> v;
            load_quad(v, src, st, i / (NS / 4), i % (NS / 4));
            store_quad(v, at, stride, i / (NS / 4), i % (NS / 4));
        }
    };
    // x and dy of a head: half the workgroup each
    constexpr int XB = (L / 4) * (P / 4), XPER = (XB + 255) / 256;
    quad<TI> raw[XPER];
    auto fetch_xy = [&](int h) {
        const bool y = wave >= 4;
        const TI *src = y ? static_cast<const TI *>(a.d_y) + (flat0 * p.H + h) * P : xb + static_cast<int64_t>(h) * P;
        const int64_t st = y ? static_cast<int64_t>(p.H) * P : p.x_st;
#pragma unroll
        for (int k = 0; k < XPER; ++k) {
            const int i = (tid & 255) + 256 * k;
            if (XB % 256 == 0 || i < XB) load_quad(raw[k], src, st, i / (P / 4), i % (P / 4));
        }
    };
    auto store_xy = [&] {
#pragma unroll
        for (int k = 0; k < XPER; ++k) {
            const int i = (tid & 255) + 256 * k;
            if (XB % 256 == 0 || i < XB) store_quad(raw[k], wave >= 4 ? Cf::YN : Cf::XN, RP, i / (P / 4), i % (P / 4));
        }
    };
    // columns past d_state and d_head, the score tiles above the diagonal and
    // the sums no tile writes stay zero
    for (int i = tid; i < Cf::END / 2; i += 512) reinterpret_cast<uint32_t *>(lds)[i] = 0;
    for (int i = tid; i < Cf::FEND; i += 512) fl[i] = 0.f;
    lds_barrier();
    stage(Cf::BN, RN, bb, p.b_st);
    stage(Cf::CN, RN, cb, p.c_st);
    lds_barrier();

    constexpr int TILES = ST * (ST + 1) / 2, MT = (TILES + 7) / 8;
    f32x4 K[MT];  // scores of this wave's tiles: rows s, columns t
    int tile_i[MT], tile_j[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        K[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        int ti = 0, tj = wave + 8 * m;
        tile_i[m] = -1;
        if (tj >= TILES) continue;
        while (tj > ti) { tj -= ti + 1; ++ti; }
        tile_i[m] = ti;
        tile_j[m] = tj;
        for (int kk = 0; kk < NKS; ++kk) {
            parts8<EX> u, v;
#pragma unroll
            for (int part = 0; part < EX; ++part) {
                load_rows(u.f[part], lds + Cf::BN + part * L * RN, RN, 16 * tj, kk, g, c16);
                load_rows(v.f[part], lds + Cf::CN + part * L * RN, RN, 16 * ti, kk, g, c16);
            }
            mfma_parts<EX, EX, ORD>(K[m], u, v);
        }
    }
    // this wave's 16 columns of B and C with the tokens as contraction; slot
    // (s % 2) 4 + r of step s / 2 is the element of row 16 s + 4 g + r
    const bool rows_on = wave < NT;
    const int n0 = (rows_on ? wave : 0) * 16;
    parts8<EX> Bt[TK], Ct[TK];
#pragma unroll
    for (int ks = 0; ks < TK; ++ks)
#pragma unroll
        for (int part = 0; part < EX; ++part) {
            load_cols(Bt[ks].f[part], lds + Cf::BN + part * L * RN, RN, 32 * ks, n0, g, c16);
            load_cols(Ct[ks].f[part], lds + Cf::CN + part * L * RN, RN, 32 * ks, n0, g, c16);
        }
    auto elem = [&](const parts8<EX> (&f)[TK], int s, int r) {
        float v = 0.f;
#pragma unroll
        for (int part = EX - 1; part >= 0; --part) v += bf16_to_f32(f[s / 2].f[part].s[(s % 2) * 4 + r]);
        return v;
    };
    f32x4 dCs[ST], dBs[ST];  // sums over the heads: rows 16 s + 4 g + r, column n0 + c16
#pragma unroll
    for (int s = 0; s < ST; ++s) dCs[s] = dBs[s] = f32x4{0.f, 0.f, 0.f, 0.f};

    // this wave's rows of both states, channels in the operand's slot order
    f32x4 Sv[PKS][2], Gv[PKS][2];
    auto fetch_states = [&](int h) {
        const int64_t so = ((static_cast<int64_t>(item) * p.H + h) * NS + n0) * P;
#pragma unroll
        for (int ks = 0; ks < PKS; ++ks)
#pragma unroll
            for (int hq = 0; hq < 2; ++hq) {
                const int c = 32 * ks + 16 * hq + 4 * g;
                Sv[ks][hq] = Gv[ks][hq] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (rows_on && (P >= 32 || hq == 0)) {
                    Sv[ks][hq] = *reinterpret_cast<const f32x4 *>(a.states + so + static_cast<uint32_t>(c16 * P + c));
                    Gv[ks][hq] = *reinterpret_cast<const f32x4 *>(a.gstates + so + static_cast<uint32_t>(c16 * P + c));
                }
            }
    };
    float rawdt = 0.f;  // wave 7: one token a lane
    auto fetch_dt = [&](int h) {
        if (wave == 7 && lane < len) rawdt = io<TI>::ld(static_cast<const TI *>(p.dt), (flat0 + lane) * p.H + h);
    };
    fetch_xy(h0);
    fetch_states(h0);
    fetch_dt(h0);
    for (int h = h0; h < h1; ++h) {
        // what follows from the lane's place is computed again for every head:
        // kept over the loop it would push the tiles out of the registers
        asm volatile("" : "+v"(tid), "+v"(lane), "+v"(g), "+v"(c16));
        // ---- x, dy and the decays into LDS; the next head's x and dy on their way
        store_xy();
        const float A = p.A[h];
        float raw_dt = 0.f, dt = 0.f, tot = 0.f;
        bool gone = false;  // the token ends everything before it (kGone)
        if (wave == 7) {
            raw_dt = rawdt + (p.dt_bias ? p.dt_bias[h] : 0.f);
            dt = p.softplus ? softplus_rel(raw_dt) : raw_dt;
            if (lane >= len) dt = 0.f;
            // D compares sums over the rest of the chunk whose difference may
            // be one token's log: kept in 64 bits, as two floats in LDS
            double sum = static_cast<double>(A) * 1.4426950408889634 * dt;
            gone = sum < kGone;
            if (gone) sum = kGone;
            const float la = static_cast<float>(sum);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_down(sum, d);
                if (lane + d < 64) sum += o;
            }
            tot = static_cast<float>(__shfl(sum, 0));
            double rest = __shfl_down(sum, 1);
            if (lane == 63) rest = 0.0;
            const float suf = static_cast<float>(rest);
            const float ecum = fast_exp2(lane_scan(la));
            if (lane < L) {
                fl[Cf::FDT + lane] = dt;
                fl[Cf::FSUF + lane] = suf;
                fl[Cf::FLO + lane] = static_cast<float>(rest - suf);
                fl[Cf::FCUM + lane] = ecum;
                fl[Cf::FWS + lane] = fast_exp2(suf);
            }
        }
        if (h + 1 < h1) {
            fetch_xy(h + 1);
            fetch_dt(h + 1);
        }
        lds_barrier();

        // ---- causal tiles of Q; M1 = Q D dt_s, M2 = K D into LDS; sums of E
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int ti = tile_i[m], tj = tile_j[m];
            if (ti < 0) continue;
            f32x4 q = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < PKS; ++kk) {
                parts8<EX> u, v;
#pragma unroll
                for (int part = 0; part < EX; ++part) {
                    load_rows(u.f[part], lds + Cf::XN + part * L * RP, RP, 16 * tj, kk, g, c16);
                    load_rows(v.f[part], lds + Cf::YN + part * L * RP, RP, 16 * ti, kk, g, c16);
                }
                mfma_parts<EX, EX, ORD>(q, u, v);
            }
            const int t = 16 * ti + c16, s0 = 16 * tj + 4 * g;
            const float suf_t = fl[Cf::FSUF + t];
            const f32x4 suf_s = *reinterpret_cast<const f32x4 *>(fl + Cf::FSUF + s0);
            const float lo_t = fl[Cf::FLO + t];
            const f32x4 lo_s = *reinterpret_cast<const f32x4 *>(fl + Cf::FLO + s0);
            const f32x4 dt_s = *reinterpret_cast<const f32x4 *>(fl + Cf::FDT + s0);
            double rowsum = 0.0, E[4];  // the sums' difference is wanted: their own rounding would show
            granule m1[XP], m2[XP];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = s0 + r <= t ? fast_exp2((suf_s[r] - suf_t) + (lo_s[r] - lo_t)) : 0.f;
                const float qd = q[r] * d, kd = K[m][r] * d;
                E[r] = static_cast<double>(q[r]) * kd;
                // the diagonal passes through no token's decay: kept apart, it
                // would only leave its rounding in the difference of the sums
                if (s0 + r == t) {
                    fl[Cf::FQD + t] = q[r];
                    fl[Cf::FED + t] = static_cast<float>(E[r]);
                    E[r] = 0.0;
                }
                rowsum = fma(E[r], static_cast<double>(dt_s[r]), rowsum);
                float v1 = qd * dt_s[r], v2 = kd;
#pragma unroll
                for (int part = 0; part < XP; ++part) {
                    m1[part].s[r] = f32_to_bf16(v1);
                    m2[part].s[r] = f32_to_bf16(v2);
                    v1 -= bf16_to_f32(m1[part].s[r]);
                    v2 -= bf16_to_f32(m2[part].s[r]);
                }
            }
#pragma unroll
            for (int part = 0; part < XP; ++part) {
                *reinterpret_cast<uint2 *>(lds + Cf::M1 + part * L * RL + t * RL + col_pos(s0)) = m1[part].u;
                *reinterpret_cast<uint2 *>(lds + Cf::M2 + part * L * RL + t * RL + col_pos(s0)) = m2[part].u;
            }
            rowsum += __shfl_xor(rowsum, 16);
            rowsum += __shfl_xor(rowsum, 32);
            if (g == 0) rsum[tj * L + t] = rowsum;
            const double colsum = sum16<4, 8>(E, c16);
            if (c16 % 4 == 0) csum[ti * L + s0 + c16 / 4] = colsum;
        }

        // ---- the states' shares of dC and dB, and their sums with C and B
        if (rows_on) {
            float gs = 0.f;
            f32x4 ts[ST], tg[ST];
#pragma unroll
            for (int s = 0; s < ST; ++s) ts[s] = tg[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < PKS; ++ks) {
                parts8<SP> Sf, Gf;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    gs = fmaf(Sv[ks][j / 4][j % 4], Gv[ks][j / 4][j % 4], gs);
                    split_to<SP>(Sf, j, Sv[ks][j / 4][j % 4]);
                    split_to<SP>(Gf, j, Gv[ks][j / 4][j % 4]);
                }
                if (Cf::GLDS)
#pragma unroll
                    for (int part = 0; part < XP; ++part)
                        *reinterpret_cast<uint4 *>(lds + Cf::GN + part * NS * RP + (n0 + c16) * RP + 32 * ks + 8 * g) = Gf.f[part].u;
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    parts8<EX> y, x;
#pragma unroll
                    for (int part = 0; part < EX; ++part) {
                        load_rows(y.f[part], lds + Cf::YN + part * L * RP, RP, 16 * s, ks, g, c16);
                        load_rows(x.f[part], lds + Cf::XN + part * L * RP, RP, 16 * s, ks, g, c16);
                    }
                    mfma_parts<EX, SP, 3>(ts[s], y, Sf);
                    mfma_parts<EX, SP, 3>(tg[s], x, Gf);
                }
            }
            if (h + 1 < h1) fetch_states(h + 1);
            gs = lane_scan(gs);
            if (lane == 63) fl[Cf::FX + wave] = gs;
            float vi[4 * ST], vo[4 * ST];
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                const f32x4 cum = *reinterpret_cast<const f32x4 *>(fl + Cf::FCUM + 16 * s + 4 * g);
                const f32x4 ws = *reinterpret_cast<const f32x4 *>(fl + Cf::FWS + 16 * s + 4 * g);
                const f32x4 dts = *reinterpret_cast<const f32x4 *>(fl + Cf::FDT + 16 * s + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ts[s][r] *= cum[r];
                    tg[s][r] *= ws[r];
                    vi[4 * s + r] = ts[s][r] * elem(Ct, s, r);
                    vo[4 * s + r] = tg[s][r] * elem(Bt, s, r);
                    dCs[s][r] += ts[s][r];
                    dBs[s][r] = fmaf(dts[r], tg[s][r], dBs[s][r]);
                }
            }
            const float si = sum16<4 * ST, 8>(vi, c16), sg = sum16<4 * ST, 8>(vo, c16);
            const int k = c16 / (4 / ST), t = 16 * (k / 4) + 4 * g + k % 4;
            if (c16 % (4 / ST) == 0) {
                fl[Cf::FI + wave * L + t] = si;
                fl[Cf::FO + wave * L + t] = sg;
            }
        }
        lds_barrier();

        // ---- the chunk's own shares of dC and dB
        if (rows_on) {
#pragma unroll
            for (int s = 0; s < ST; ++s) {
#pragma unroll
                for (int ks = 0; ks <= s / 2; ++ks) {
                    parts8<XP> m;
#pragma unroll
                    for (int part = 0; part < XP; ++part) load_rows(m.f[part], lds + Cf::M1 + part * L * RL, RL, 16 * s, ks, g, c16);
                    mfma_parts<XP, EX, ORD>(dCs[s], m, Bt[ks]);
                }
#pragma unroll
                for (int ks = s / 2; ks < TK; ++ks) {
                    parts8<XP> m;
#pragma unroll
                    for (int part = 0; part < XP; ++part) load_cols(m.f[part], lds + Cf::M1 + part * L * RL, RL, 32 * ks, 16 * s, g, c16);
                    mfma_parts<XP, EX, ORD>(dBs[s], m, Ct[ks]);
                }
            }
        }
        // ---- du and dx: 16 x 16 tiles (strip s, channel tile pt)
        const float Dh = p.D ? p.D[h] : 0.f;
#pragma unroll 1
        for (int u = wave; u < PT * ST; u += 8) {
            const int pt = u % PT, s = u / PT;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            const float *Gp = a.gstates + (static_cast<int64_t>(item) * p.H + h) * NS * P + 16 * pt;
#pragma unroll
            for (int kk = 0; kk < NKS; ++kk) {
                parts8<XP> gf;
                if constexpr (Cf::GLDS && NS >= 32) {
#pragma unroll
                    for (int part = 0; part < XP; ++part)
                        load_cols(gf.f[part], lds + Cf::GN + part * NS * RP, RP, 32 * kk, 16 * pt, g, c16);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        split_to<XP>(gf, j, NS >= 32 || j < 4 ? Gp[static_cast<uint32_t>((32 * kk + kperm(g, j)) * P + c16)] : 0.f);
                }
                parts8<EX> b;
#pragma unroll
                for (int part = 0; part < EX; ++part) load_rows(b.f[part], lds + Cf::BN + part * L * RN, RN, 16 * s, kk, g, c16);
                mfma_parts<EX, XP, ORD>(acc, b, gf);
            }
            acc *= *reinterpret_cast<const f32x4 *>(fl + Cf::FWS + 16 * s + 4 * g);
            const f32x4 dts = *reinterpret_cast<const f32x4 *>(fl + Cf::FDT + 16 * s + 4 * g);
            float dyv[4] = {};
#pragma unroll
            for (int ks = 0; ks < TK; ++ks) {
                if (ks < s / 2) continue;
                parts8<EX> y;
                parts8<XP> m;
#pragma unroll
                for (int part = 0; part < EX; ++part) load_cols(y.f[part], lds + Cf::YN + part * L * RP, RP, 32 * ks, 16 * pt, g, c16);
#pragma unroll
                for (int part = 0; part < XP; ++part) load_cols(m.f[part], lds + Cf::M2 + part * L * RL, RL, 32 * ks, 16 * s, g, c16);
                mfma_parts<XP, EX, ORD>(acc, m, y);
                if (ks == s / 2)
#pragma unroll
                    for (int part = EX - 1; part >= 0; --part)
#pragma unroll
                        for (int r = 0; r < 4; ++r) dyv[r] += bf16_to_f32((s & 1) ? y.f[part].s[4 + r] : y.f[part].s[r]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * s + 4 * g + r;
                if (len == L || t < len)
                    io<TI>::st(static_cast<TI *>(a.dx) + ((flat0 + 16 * s + r) * p.H + h) * P + 16 * pt,
                               static_cast<uint32_t>(4 * g * p.H * P + c16), fmaf(dts[r], acc[r], Dh * dyv[r]));
            }
        }
        // ---- the step sizes: one token a lane
        if (wave == 7) {
            double R = 0.0, Cs = 0.0;
            float in = 0.f, out = 0.f, X = 0.f;
            if (lane < L) {
#pragma unroll
                for (int k = 0; k < ST; ++k) {
                    R += rsum[k * L + lane];
                    Cs += csum[k * L + lane];
                }
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    in += fl[Cf::FI + k * L + lane];
                    out += fl[Cf::FO + k * L + lane];
                }
            }
#pragma unroll
            for (int k = 0; k < NT; ++k) X += fl[Cf::FX + k];
            const float o = dt * out;
            double left = R - dt * Cs + in, right = o;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double l = __shfl_down(left, d), r = __shfl_up(right, d);
                if (lane + d < 64) left += l;
                if (lane >= d) right += r;
            }
            right = __shfl_up(right, 1);
            if (lane == 0) right = 0.0;
            // nothing passes through a token that is gone; what its sums leave is
            // their rounding, and it would meet the huge step in dA
            const double dlog = gone ? 0.0 : left + right + static_cast<double>(fast_exp2(tot)) * X;
            float dd = static_cast<float>(Cs + (lane < L ? fl[Cf::FED + lane] : 0.f) + out + A * dlog);
            if (p.softplus) dd *= sigmoid_f32(raw_dt);
            if (lane >= len) dd = 0.f;
            if (lane < len) io<TI>::st(static_cast<TI *>(a.ddt), (flat0 + lane) * p.H + h, dd);
            const float sa = lane_scan(static_cast<float>(dt * dlog)), sd = lane_scan(lane < L ? fl[Cf::FQD + lane] : 0.f);
            const float sb = lane_scan(dd);
            if (lane == 63) {
                a.scalars[(0 * static_cast<int64_t>(p.H) + h) * items + item] = sa;
                a.scalars[(1 * static_cast<int64_t>(p.H) + h) * items + item] = sd;
                a.scalars[(2 * static_cast<int64_t>(p.H) + h) * items + item] = sb;
            }
        }
        lds_barrier();  // the next head's tiles may be written
    }
    if (rows_on)
#pragma unroll
        for (int s = 0; s < ST; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * s + 4 * g + r;
                if (t >= len) continue;
                const int64_t at = ((flat0 + t) * p.G + grp) * NS + n0 + c16;
                if (a.part_B) {
                    const int64_t plane = static_cast<int64_t>(p.B) * p.T * p.G * NS;
                    a.part_B[split * plane + at] = dBs[s][r];
                    a.part_C[split * plane + at] = dCs[s][r];
                } else {
                    io<TI>::st(static_cast<TI *>(a.dB), at, dBs[s][r]);
                    io<TI>::st(static_cast<TI *>(a.dC), at, dCs[s][r]);
                }
            }
}

// dB and dC from the splits' sums, 4 values a thread
template <typename TI>
__global__ void __launch_bounds__(256) ssm_grad_sum_kernel(SsmGrad a, int64_t plane) {
    if (a.q.p.cu_seqlens && *a.q.status != 0) return;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= 2 * plane) return;
    const float *src = i < plane ? a.part_B + i : a.part_C + (i - plane);
    TI *dst = i < plane ? static_cast<TI *>(a.dB) + i : static_cast<TI *>(a.dC) + (i - plane);
    f32x4 v = *reinterpret_cast<const f32x4 *>(src);
    for (int k = 1; k < a.splits; ++k) v += *reinterpret_cast<const f32x4 *>(src + k * plane);
#pragma unroll
    for (int c = 0; c < 4; ++c) io<TI>::st(dst, c, v[c]);
}

template <typename TI, int NS, int P>
hipError_t grad_run(const SsmGrad &a, hipStream_t s) {
    const int64_t items = a.q.p.cu_seqlens ? static_cast<int64_t>(a.q.chunks_per_seq) + a.q.p.N
                                           : static_cast<int64_t>(a.q.p.N) * a.q.chunks_per_seq;
    const int64_t want = items * GradCfg<TI, NS, P>::SUB * a.q.p.G * a.splits;
    if (want == 0) return hipSuccess;
    hipLaunchKernelGGL((ssm_grad_kernel<TI, NS, P>), dim3(static_cast<unsigned>((want + 7) / 8 * 8)), dim3(512), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part_B || a.q.p.T == 0) return e;
    const int64_t plane = static_cast<int64_t>(a.q.p.B) * a.q.p.T * a.q.p.G * NS;
    hipLaunchKernelGGL((ssm_grad_sum_kernel<TI>), dim3(static_cast<unsigned>((2 * plane / 4 + 255) / 256)), dim3(256), 0, s, a, plane);
    return hipGetLastError();
}
template <typename TI, int NS>
hipError_t grad_p(const SsmGrad &a, hipStream_t s) {
    switch (a.q.p.P) {
        case 16: return grad_run<TI, NS, 16>(a, s);
        case 32: return grad_run<TI, NS, 32>(a, s);
        case 64: return grad_run<TI, NS, 64>(a, s);
        default: return grad_run<TI, NS, 128>(a, s);
    }
}
template <typename TI>
hipError_t grad_n(const SsmGrad &a, hipStream_t s) {
    switch (a.q.p.Ns) {
        case 16: return grad_p<TI, 16>(a, s);
        case 32: return grad_p<TI, 32>(a, s);
        case 64: return grad_p<TI, 64>(a, s);
        default: return grad_p<TI, 128>(a, s);
    }
}

}  // namespace
}  // namespace kda
