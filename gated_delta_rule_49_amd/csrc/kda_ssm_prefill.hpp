// The selective state space scan over whole sequences; the chunked form is in
// kda_ssm_scan.hpp.
//
// A wave owns PW = 32 channels of one head: the state [d_state, 32] stays in
// matrix-core accumulators over the whole walk, x is loaded straight into
// operand order (a lane takes neighbouring channels of the rows its operand
// slots need, so neither x nor y passes through LDS), and the accumulators of
// the state turn into the operand of C S without a lane exchange.  The waves
// of a workgroup own heads of one group and share the chunk's B, C and causal
// scores in LDS.
//
// One sequence with few heads does not fill 256 CUs: it is cut into segments.
// Phase 1 runs the state part alone over every segment but the last, from
// zero; a small kernel chains the segments' end states; phase 2 runs the full
// scan over all segments at once.
#pragma once
#include "kda_ssm_scan.hpp"

namespace kda {

namespace {

template <typename TI, typename TO, int NS, int PW, int NW, int MODE>
struct ScanCfg {
    static constexpr bool BF = std::is_same<TI, bf16_t>::value, FULL = MODE == SSM_FULL;
    static constexpr int EX = quad<TI>::PARTS;            // parts of an input
    static constexpr int L = BF ? 64 : 32;                // tokens of a chunk
    static constexpr int ORD = BF ? 2 : 3;
    static constexpr int XP = 3;                          // parts of w x: the state keeps fp32 accuracy
    static constexpr int GP = BF ? 2 : 3;                 // parts of the scores
    // the state as an operand of C S: a bf16 y carries a rounding of up to
    // 2^-9 of its own; one part of S adds an error of that size only to what
    // the state contributes
    static constexpr int SP = !BF ? 3 : std::is_same<TO, bf16_t>::value ? 1 : 2;
    static constexpr int NT = NS / 16, KS = (NS + 31) / 32, NK = KS * 32;
    static constexpr int CT = PW / 16, ST = L / 16, TK = L / 32;
    static constexpr int RN = NK + 8, RT = L + 8;         // LDS row strides: 16-byte pieces of 16 rows hit all banks
    static constexpr int NBUF = BF ? 2 : 1;
    static constexpr int CN = FULL ? EX * L * RN : 0;     // C, and B by rows
    static constexpr int BT = EX * NS * RT;               // B transposed
    static constexpr int GT = FULL ? GP * L * RT : 0;     // causal scores
    static constexpr int BUF = 2 * CN + BT + GT;
    static constexpr int WV = 4 * L;                      // per wave: w, row factor, suf, dt
    static constexpr size_t BYTES = sizeof(bf16_t) * NBUF * BUF + sizeof(float) * NW * WV;
};

template <typename TI, typename TO, int NS, int PW, int NW, int MODE>
__global__ void __launch_bounds__(64 * NW) ssm_scan_kernel(SsmScan q, int blocks_per_group, int phase) {
    using Cf = ScanCfg<TI, TO, NS, PW, NW, MODE>;
    constexpr int EX = Cf::EX, L = Cf::L, ORD = Cf::ORD, XP = Cf::XP, GP = Cf::GP, SP = Cf::SP, NT = Cf::NT, KS = Cf::KS;
    constexpr int CT = Cf::CT, ST = Cf::ST, TK = Cf::TK, RN = Cf::RN, RT = Cf::RT, NBUF = Cf::NBUF;
    constexpr bool FULL = MODE == SSM_FULL, REV = MODE == SSM_REVERSE;
    __shared__ __attribute__((aligned(16))) char smem[Cf::BYTES];
    const SsmParams &p = q.p;
    if (q.user_status && !p.cu_seqlens && phase == 2 && blockIdx.x == 0 && threadIdx.x == 0) *q.user_status = 0;
    const int block = xcd_order(blockIdx.x, gridDim.x);
    const int x_seg = block / (p.G * blocks_per_group);
    if (x_seg >= q.segs_bound) return;
    const SsmSeg sg = ssm_seg(q, x_seg);
    if (!sg.valid) return;
    // the last segment's end state is nobody's entering state (reverse: the first's)
    if (phase == 1 && (REV ? sg.s == 0 : sg.s == sg.count - 1)) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c16 = lane & 15;
    const int grp = (block / blocks_per_group) % p.G, hpg = p.H / p.G, cb_n = p.P / PW;
    const int item = (block % blocks_per_group) * NW + wave;
    const bool on = item < hpg * cb_n;               // waves past the group's heads only stage
    const int h = grp * hpg + (on ? item / cb_n : 0);
    const int pc = (on ? item % cb_n : 0) * PW + c16 * CT;  // the lane's channels pc .. pc + CT - 1

    bf16_t *lds = reinterpret_cast<bf16_t *>(smem);
    float *wv = reinterpret_cast<float *>(smem + sizeof(bf16_t) * NBUF * Cf::BUF) + wave * Cf::WV;
    float *fv = wv + L, *sv = wv + 2 * L, *dv = wv + 3 * L;
    auto Cn = [&](int b, int part) { return lds + b * Cf::BUF + part * L * RN; };
    auto Bn = [&](int b, int part) { return lds + b * Cf::BUF + Cf::CN + part * L * RN; };
    auto Bt = [&](int b, int part) { return lds + b * Cf::BUF + 2 * Cf::CN + part * NS * RT; };
    auto Gt = [&](int b, int part) { return lds + b * Cf::BUF + 2 * Cf::CN + Cf::BT + part * L * RT; };

    const int64_t flat0 = static_cast<int64_t>(sg.row) * p.T + sg.t0;
    const int64_t per_head = static_cast<int64_t>(NS) * p.P;
    const TI *xb = static_cast<const TI *>(p.x) + sg.row * p.x_sb + sg.t0 * p.x_st + static_cast<int64_t>(h) * p.P + pc;
    const TI *bb = static_cast<const TI *>(p.Bm) + sg.row * p.b_sb + sg.t0 * p.b_st + static_cast<int64_t>(grp) * NS;
    const TI *cb = static_cast<const TI *>(p.Cm) + sg.row * p.c_sb + sg.t0 * p.c_st + static_cast<int64_t>(grp) * NS;
    const TI *dtb = static_cast<const TI *>(p.dt) + flat0 * p.H + h;
    TO *yb = static_cast<TO *>(p.y) + (flat0 * p.H + h) * p.P + pc;
    const float A2 = p.A[h] * kLog2e, Dh = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;

    // the state: a lane holds rows 16 nt + 4 g + r, channels pc + ct
    f32x4 S[NT][CT];
    {
        const float *src = phase == 1 ? nullptr
                           : q.seg_state ? q.seg_state + (static_cast<int64_t>(x_seg) * p.H + h) * per_head
                           : p.initial_state ? p.initial_state + (static_cast<int64_t>(sg.n) * p.H + h) * per_head : nullptr;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                lanevec<float, CT> v;
                v.zero();
                if (src) v.ld(src + (16 * nt + 4 * g + r) * p.P + pc);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[nt][ct][r] = v.get(ct);
            }
    }
    auto store_state = [&](float *dst) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) v[ct] = S[nt][ct][r];
                lanevec<float, CT>::st(dst + (16 * nt + 4 * g + r) * p.P + pc, v);
            }
    };

    // zero what no staging writes: columns past d_state, the score tiles above the diagonal
    if (FULL) {
        if (NS < 32)
            for (int i = tid; i < NBUF * 2 * Cf::CN; i += 64 * NW) lds[(i / (2 * Cf::CN + !Cf::CN)) * Cf::BUF + i % (2 * Cf::CN + !Cf::CN)] = 0;
        for (int b = 0; b < NBUF; ++b)
            for (int i = tid; i < Cf::GT; i += 64 * NW) Gt(b, 0)[i] = 0;
        lds_barrier();
    }

    // staging of a chunk's B and C: a thread takes 4 tokens by 4 channels
    constexpr int BLOCKS = (L / 4) * (NS / 4), PER = (BLOCKS + 64 * NW - 1) / (64 * NW);
    quad<TI> rawB[PER], rawC[FULL ? PER : 1];
    auto fetch = [&](int c) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid + k * 64 * NW;
            const int tq = i / (NS / 4), nq = i % (NS / 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = c * L + tq * 4 + r;
                const bool in = i < BLOCKS && t < sg.len;
                rawB[k].zero(r);
                if (in) rawB[k].ld(r, bb + t * p.b_st + nq * 4);
                if (FULL) {
                    rawC[k].zero(r);
                    if (in) rawC[k].ld(r, cb + t * p.c_st + nq * 4);
                }
            }
        }
    };
    auto stage = [&](int b) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid + k * 64 * NW;
            const int tq = i / (NS / 4), nq = i % (NS / 4);
            if (i < BLOCKS)
#pragma unroll
                for (int part = 0; part < EX; ++part)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (FULL) {
                            *reinterpret_cast<uint2 *>(Bn(b, part) + (tq * 4 + r) * RN + col_pos(nq * 4)) = rawB[k].row(r, part).u;
                            *reinterpret_cast<uint2 *>(Cn(b, part) + (tq * 4 + r) * RN + col_pos(nq * 4)) = rawC[k].row(r, part).u;
                        }
                        *reinterpret_cast<uint2 *>(Bt(b, part) + (nq * 4 + r) * RT + col_pos(tq * 4)) = rawB[k].col(r, part).u;
                    }
        }
    };
    // causal scores of a staged chunk: tile (ti, tj) taken as B C^T, so that a
    // lane holds 4 neighbouring columns of one row
    auto scores = [&](int b) {
        for (int k = wave; k < ST * (ST + 1) / 2; k += NW) {
            int ti = 0, tj = k;
            while (tj > ti) { tj -= ti + 1; ++ti; }
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                parts8<EX> a, bf;
#pragma unroll
                for (int part = 0; part < EX; ++part) {
                    a.f[part].u = *reinterpret_cast<const uint4 *>(Bn(b, part) + (16 * tj + c16) * RN + kk * 32 + 8 * g);
                    bf.f[part].u = *reinterpret_cast<const uint4 *>(Cn(b, part) + (16 * ti + c16) * RN + kk * 32 + 8 * g);
                }
                mfma_parts<EX, EX, ORD>(acc, a, bf);
            }
            granule out[GP];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = ti == tj && 4 * g + r > c16 ? 0.f : acc[r];
#pragma unroll
                for (int part = 0; part < GP; ++part) {
                    out[part].s[r] = f32_to_bf16(v);
                    v -= bf16_to_f32(out[part].s[r]);
                }
            }
#pragma unroll
            for (int part = 0; part < GP; ++part)
                *reinterpret_cast<uint2 *>(Gt(b, part) + (16 * ti + c16) * RT + col_pos(16 * tj + 4 * g)) = out[part].u;
        }
    };
    // x (rows in the operand's slot order) and dt of a chunk
    lanevec<TI, CT> xr[TK][8], xn[TK][8];
    TI dtr = TI(0), dtn = TI(0);
    auto fetch_x = [&](int c, lanevec<TI, CT> (&xv)[TK][8], TI &d) {
#pragma unroll
        for (int ks = 0; ks < TK; ++ks)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = c * L + 32 * ks + kperm(g, j);
                xv[ks][j].zero();
                if (t < sg.len) xv[ks][j].ld(xb + t * p.x_st);
            }
        d = TI(0);
        if (lane < L && c * L + lane < sg.len) d = dtb[static_cast<int64_t>(c * L + lane) * p.H];
    };

    const int chunks = (sg.len + L - 1) / L;
    float seg_log = 0.f;
    auto order = [&](int i) { return REV ? chunks - 1 - i : i; };
    if (chunks > 0) {
        fetch(order(0));
        fetch_x(order(0), xr, dtr);
        stage(0);
        if (chunks > 1) fetch(order(1));
        lds_barrier();
        if (FULL) {
            scores(0);
            lds_barrier();
        }
    }
    for (int i = 0; i < chunks; ++i) {
        const int b = NBUF == 2 ? i & 1 : 0;
        const int t0 = order(i) * L;
        if (NBUF == 2 && i + 1 < chunks) {  // the next chunk into the other buffer
            stage(b ^ 1);
            if (i + 2 < chunks) fetch(order(i + 2));
        }
        if (i + 1 < chunks) fetch_x(order(i + 1), xn, dtn);
        if (on) {
            // the state entering the 64-token chunk (from the right in the reverse order)
            if (phase == 2 && p.chunk_states && t0 % q.state_chunk == 0)
                store_state(p.chunk_states + ((static_cast<int64_t>(sg.chunk + t0 / 64) * (64 / q.state_chunk) + t0 % 64 / q.state_chunk) * p.H + h) * per_head);
            // decays, one token a lane
            float dt = io<TI>::ld(&dtr, 0) + bias;
            if (p.softplus) dt = softplus_rel(dt);
            if (lane >= L || t0 + lane >= sg.len) dt = 0.f;
            const float la = A2 * dt;
            const float incl = suffix_sum(la, lane);
            const float tot = __shfl(incl, 0);
            const float suf = after(incl, lane);
            const bool fast = fabsf(tot) < kFastTot;
            if (lane < L) {
                if (REV) {
                    wv[lane] = fast_exp2(prefix_sum(la, lane));
                } else {
                    wv[lane] = dt * fast_exp2(suf);
                }
                if (FULL) {
                    fv[lane] = fast ? fast_exp2(-suf) : fast_exp2(prefix_sum(la, lane));
                    sv[lane] = suf;
                    dv[lane] = dt;
                }
            }
            seg_log += tot;
            wave_lds_fence();
            const float dec = fast_exp2(tot);

            parts8<XP> xw[TK][CT];
#pragma unroll
            for (int ks = 0; ks < TK; ++ks) {
                float wq[8];
#pragma unroll
                for (int hq = 0; hq < 2; ++hq) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(wv + 32 * ks + 16 * hq + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) wq[4 * hq + r] = v[r];
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int j = 0; j < 8; ++j) split_to<XP>(xw[ks][ct], j, xr[ks][j].get(ct) * wq[j]);
            }
            if (fast || !FULL)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) S[nt][ct] *= dec;
            if constexpr (FULL) {
                f32x4 acc[ST][CT];
#pragma unroll
                for (int s = 0; s < ST; ++s)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) acc[s][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
                // C S
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    parts8<SP> sf[CT];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            split_to<SP>(sf[ct], r, S[2 * kk][ct][r]);
                            split_to<SP>(sf[ct], 4 + r, 2 * kk + 1 < NT ? S[2 * kk + 1 < NT ? 2 * kk + 1 : 0][ct][r] : 0.f);
                        }
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        parts8<EX> a;
#pragma unroll
                        for (int part = 0; part < EX; ++part)
                            a.f[part].u = *reinterpret_cast<const uint4 *>(Cn(b, part) + (16 * s + c16) * RN + kk * 32 + 8 * g);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) mfma_parts<EX, SP, ORD>(acc[s][ct], a, sf[ct]);
                    }
                }
                if (fast) {
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
#pragma unroll
                        for (int ks = 0; ks <= s / 2; ++ks) {
                            parts8<GP> a;
#pragma unroll
                            for (int part = 0; part < GP; ++part)
                                a.f[part].u = *reinterpret_cast<const uint4 *>(Gt(b, part) + (16 * s + c16) * RT + ks * 32 + 8 * g);
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) mfma_parts<GP, XP, ORD>(acc[s][ct], a, xw[ks][ct]);
                        }
                        const f32x4 f = *reinterpret_cast<const f32x4 *>(fv + 16 * s + 4 * g);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) acc[s][ct] *= f;
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        const f32x4 f = *reinterpret_cast<const f32x4 *>(fv + 16 * s + 4 * g);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) acc[s][ct] *= f;
                        const int row = 16 * s + c16;
                        const float suf_row = sv[row];
#pragma unroll
                        for (int ks = 0; ks <= s / 2; ++ks) {
                            parts8<GP> m;
#pragma unroll
                            for (int part = 0; part < GP; ++part)
                                m.f[part].u = *reinterpret_cast<const uint4 *>(Gt(b, part) + row * RT + ks * 32 + 8 * g);
                            float mv[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                mv[j] = 0.f;
#pragma unroll
                                for (int part = GP - 1; part >= 0; --part) mv[j] += bf16_to_f32(m.f[part].s[j]);
                            }
#pragma unroll
                            for (int hq = 0; hq < 2; ++hq) {
                                const int col = 32 * ks + 16 * hq + 4 * g;
                                const f32x4 sc = *reinterpret_cast<const f32x4 *>(sv + col);
                                const f32x4 dc = *reinterpret_cast<const f32x4 *>(dv + col);
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const float k = col + r <= row ? dc[r] * fast_exp2(sc[r] - suf_row) : 0.f;
                                    split_to<GP>(m, 4 * hq + r, mv[4 * hq + r] * k);
                                }
                            }
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) {
                                parts8<EX> xe;
#pragma unroll
                                for (int j = 0; j < 8; ++j) split_to<EX>(xe, j, xr[ks][j].get(ct));
                                mfma_parts<GP, EX, ORD>(acc[s][ct], m, xe);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) S[nt][ct] *= dec;
                }
                // y: slot (s % 2) 4 + r of x's step s / 2 is the same row
#pragma unroll
                for (int s = 0; s < ST; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = t0 + 16 * s + 4 * g + r;
                        float v[CT];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) v[ct] = fmaf(Dh, xr[s / 2][(s % 2) * 4 + r].get(ct), acc[s][ct][r]);
                        if (t < sg.len) lanevec<TO, CT>::st(yb + static_cast<int64_t>(t) * p.H * p.P, v);
                    }
            }
            // S += B (w x)^T
#pragma unroll
            for (int ks = 0; ks < TK; ++ks)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    parts8<EX> a;
#pragma unroll
                    for (int part = 0; part < EX; ++part)
                        a.f[part].u = *reinterpret_cast<const uint4 *>(Bt(b, part) + (16 * nt + c16) * RT + ks * 32 + 8 * g);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mfma_parts<EX, XP, 3>(S[nt][ct], a, xw[ks][ct]);
                }
        }
        lds_barrier();
        if (i + 1 < chunks) {
            if (NBUF == 1) {
                stage(0);
                if (i + 2 < chunks) fetch(order(i + 2));
                lds_barrier();
            }
            if (FULL) {
                scores(NBUF == 2 ? b ^ 1 : 0);
                lds_barrier();
            }
#pragma unroll
            for (int ks = 0; ks < TK; ++ks)
#pragma unroll
                for (int j = 0; j < 8; ++j) xr[ks][j] = xn[ks][j];
            dtr = dtn;
        }
    }
    if (!on) return;
    if (phase == 1) {
        store_state(q.seg_state + (static_cast<int64_t>(x_seg) * p.H + h) * per_head);
        if (pc == 0 && g == 0) q.seg_log[static_cast<int64_t>(x_seg) * p.H + h] = seg_log;
    } else if (p.final_state && (REV ? sg.s == 0 : sg.s == sg.count - 1)) {
        store_state(p.final_state + (static_cast<int64_t>(sg.n) * p.H + h) * per_head);
    }
}

template <typename TI, typename TO, int NS, int PW, int MODE>
hipError_t run(const SsmScan &q, const SsmPlan &plan, int phase, hipStream_t s) {
    const int64_t want = static_cast<int64_t>(plan.segs_bound) * q.p.G * plan.blocks_per_group;
    const unsigned grid = static_cast<unsigned>((want + 7) / 8 * 8);
    if (plan.waves == 8)
        hipLaunchKernelGGL((ssm_scan_kernel<TI, TO, NS, PW, 8, MODE>), dim3(grid), dim3(512), 0, s, q, plan.blocks_per_group, phase);
    else
        hipLaunchKernelGGL((ssm_scan_kernel<TI, TO, NS, PW, 4, MODE>), dim3(grid), dim3(256), 0, s, q, plan.blocks_per_group, phase);
    return hipGetLastError();
}
template <typename TI, typename TO, int NS>
hipError_t run_p(const SsmScan &q, const SsmPlan &plan, int mode, int phase, hipStream_t s) {
    if (q.p.P == 16) {
        if (mode == SSM_FULL) return run<TI, TO, NS, 16, SSM_FULL>(q, plan, phase, s);
        if (mode == SSM_STATES) return run<TI, float, NS, 16, SSM_STATES>(q, plan, phase, s);
        return run<TI, float, NS, 16, SSM_REVERSE>(q, plan, phase, s);
    }
    if (mode == SSM_FULL) return run<TI, TO, NS, 32, SSM_FULL>(q, plan, phase, s);
    if (mode == SSM_STATES) return run<TI, float, NS, 32, SSM_STATES>(q, plan, phase, s);
    return run<TI, float, NS, 32, SSM_REVERSE>(q, plan, phase, s);
}
}  // namespace

template <typename TI, typename TO>
hipError_t ssm_phase(const SsmScan &q, const SsmPlan &plan, int mode, int phase, hipStream_t s) {
    switch (q.p.Ns) {
        case 16: return run_p<TI, TO, 16>(q, plan, mode, phase, s);
        case 32: return run_p<TI, TO, 32>(q, plan, mode, phase, s);
        case 64: return run_p<TI, TO, 64>(q, plan, mode, phase, s);
        default: return run_p<TI, TO, 128>(q, plan, mode, phase, s);
    }
}

}  // namespace kda
