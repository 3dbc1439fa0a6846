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
//
// 32768 tokens, 64 heads of 64 channels in 8 groups, d_state 128, bf16: phase 1
// 133 to 142 us, the chain 14, phase 2 329 to 354 (315 to 330 where no head's decay
// is wide); the bytes alone would take 131.  Phase 2 spends 51 % of its cycles
// issuing vector instructions (splitting fp32 values into bf16 parts, scaling,
// rounding) and 37 % in matrix instructions; the two overlap only between the two
// waves of a SIMD, which the barriers hold at the same place.  It spills 24
// registers.  One part of the state behind y and 32-bit sums of the logs took 293
// to 308 us, and were wrong (ScanCfg, kda_ssm_scan.hpp).  An fp32 y takes 415 to
// 425 us, fp32 inputs 1.7 times as long as bf16 ones in all.  Workgroups of 4
// waves, twice as many to a CU, move B twice and gain nothing (140 against 131 us
// for phase 1); 16 waves of 16 channels spill (520 us for phase 2).
#pragma once
#include "kda_ssm_scan.hpp"

namespace kda {

namespace {

template <typename TI, typename TO, int NS, int PW, int NW, int MODE>
struct ScanCfg {
    static constexpr bool BF = std::is_same<TI, bf16_t>::value, FULL = MODE == SSM_FULL;
    static constexpr int EX = quad<TI>::PARTS;            // parts of an input
    static constexpr int L = BF ? 64 : 32;                // tokens of a chunk
    // Parts of an fp32 operand of y's products, and the products of parts that are
    // kept (orders adding up to less than ORD).  Three hold all 24 bits and leave
    // 2^-20 of a term out: for fp32 inputs or an fp32 y.  A bf16 y between bf16
    // inputs takes two: cut off after 16 bits, a term is off by at most 2^-14, a
    // 64th of y's own half step.  (One part of the state is not enough: each of
    // d_state terms is then off by up to 2^-8, and where they cancel y is off by
    // several of its steps.)
    static constexpr int ORD = BF && std::is_same<TO, bf16_t>::value ? 2 : 3;
    static constexpr int XP = 3;                          // parts of w x: the state keeps fp32 accuracy
    static constexpr int GP = ORD, SP = ORD;              // parts of the scores, of the state in C S
    static constexpr int NT = NS / 16, KS = (NS + 31) / 32, NK = KS * 32;
    static constexpr int CT = PW / 16, ST = L / 16, TK = L / 32;
    // LDS row strides: 16-byte pieces of 16 rows hit all banks (C, scores);
    // 4 rows of transposed 8-byte pieces are 16 banks apart (B)
    static constexpr int RN = NK + 8, RT = L + 8, RB = NK / 32 % 2 ? NK : NK + 32;
    static constexpr int NBUF = BF ? 2 : 1;
    static constexpr int BN = EX * L * RB, CN = EX * L * RN;
    static constexpr int GT = FULL ? GP * L * RT : 0;     // causal scores
    static constexpr int BUF = BN + (FULL ? CN : 0) + GT;
    static constexpr int WV = (FULL ? 5 : 1) * L;         // per wave: w, row factor, suf, dt, suf's rounding
    static constexpr size_t BYTES = sizeof(bf16_t) * NBUF * BUF + sizeof(float) * NW * WV;
};

// number: this workgroup's, among `blocks`
template <typename TI, typename TO, int NS, int PW, int NW, int MODE>
__device__ __forceinline__ void ssm_scan(char *smem, const SsmScan &q, int number, int blocks, int blocks_per_group, int phase) {
    using Cf = ScanCfg<TI, TO, NS, PW, NW, MODE>;
    constexpr int EX = Cf::EX, L = Cf::L, ORD = Cf::ORD, XP = Cf::XP, GP = Cf::GP, SP = Cf::SP, NT = Cf::NT, KS = Cf::KS;
    constexpr int CT = Cf::CT, ST = Cf::ST, TK = Cf::TK, RN = Cf::RN, RB = Cf::RB, RT = Cf::RT, NBUF = Cf::NBUF;
    constexpr bool FULL = MODE == SSM_FULL, REV = MODE == SSM_REVERSE;
    const SsmParams &p = q.p;
    if (q.user_status && !p.cu_seqlens && phase == 2 && number == 0 && threadIdx.x == 0) *q.user_status = 0;
    const int block = xcd_order(number, blocks);
    const int x_seg = block / (p.G * blocks_per_group);
    if (x_seg >= q.segs_bound) return;
    const SsmSeg sg = ssm_seg(q, x_seg);
    if (!sg.valid) return;
    // the last segment's end state is nobody's entering state (reverse: the first's)
    if (phase == 1 && (REV ? sg.s == 0 : sg.s == sg.count - 1)) return;

    int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int g = lane >> 4, c16 = lane & 15;
    const int grp = (block / blocks_per_group) % p.G, hpg = p.H / p.G, cb_n = p.P / PW;
    const int item = (block % blocks_per_group) * NW + wave;
    const bool on = item < hpg * cb_n;               // waves past the group's heads only stage
    const int h = grp * hpg + (on ? item / cb_n : 0);
    const int pw0 = (on ? item % cb_n : 0) * PW;     // first channel of the wave
    const int pc = pw0 + c16 * CT;                   // the lane's channels pc .. pc + CT - 1

    bf16_t *lds = reinterpret_cast<bf16_t *>(smem);
    float *wv = reinterpret_cast<float *>(smem + sizeof(bf16_t) * NBUF * Cf::BUF) + wave * Cf::WV;
    float *fv = wv + L, *sv = wv + 2 * L, *dv = wv + 3 * L, *sl = wv + 4 * L;
    auto Bn = [&](int b, int part) { return lds + b * Cf::BUF + part * L * RB; };
    auto Cn = [&](int b, int part) { return lds + b * Cf::BUF + Cf::BN + part * L * RN; };
    auto Gt = [&](int b, int part) { return lds + b * Cf::BUF + Cf::BN + Cf::CN + part * L * RT; };

    // Uniform bases; a lane adds a 32-bit byte offset (strides are below 2^23
    // elements, so a chunk's rows stay below 2^31 bytes).
    const int64_t flat0 = static_cast<int64_t>(sg.row) * p.T + sg.t0;
    const int64_t per_head = static_cast<int64_t>(NS) * p.P;
    const TI *xb = static_cast<const TI *>(p.x) + sg.row * p.x_sb + sg.t0 * p.x_st + static_cast<int64_t>(h) * p.P + pw0;
    const TI *bb = static_cast<const TI *>(p.Bm) + sg.row * p.b_sb + sg.t0 * p.b_st + static_cast<int64_t>(grp) * NS;
    const TI *cb = static_cast<const TI *>(p.Cm) + sg.row * p.c_sb + sg.t0 * p.c_st + static_cast<int64_t>(grp) * NS;
    const TI *dtb = static_cast<const TI *>(p.dt) + flat0 * p.H + h;
    TO *yb = static_cast<TO *>(p.y) + (flat0 * p.H + h) * p.P + pw0;
    const uint32_t x_st = static_cast<uint32_t>(p.x_st), y_st = static_cast<uint32_t>(p.H) * p.P;
    const float A2 = p.A[h] * kLog2e, Dh = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;

    // the state: a lane holds rows 16 nt + 4 g + r, channels pc + ct
    f32x4 S[NT][CT];
    {
        const float *src = phase == 1 ? nullptr
                           : q.seg_state ? q.seg_state + (static_cast<int64_t>(x_seg) * p.H + h) * per_head + pw0
                           : p.initial_state ? p.initial_state + (static_cast<int64_t>(sg.n) * p.H + h) * per_head + pw0 : nullptr;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) S[nt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (src)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                lanevec<float, CT> v;
                v.ld(lane_at(src + (16 * nt + r) * p.P, 4 * g * p.P + c16 * CT));
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[nt][ct][r] = v.get(ct);
            }
    }
    // The state is kept as S 2^level: a chunk adds its tot to the level (in 64
    // bits) and scales its own w x to match, and S is multiplied out only when
    // the level has gone far, or before a store.  A chunk of a wide decay takes
    // half of it as the level, so that its own factors lie around 1.
    double level = 0.0;
    auto scale_state = [&](float f) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) S[nt][ct] *= f;
    };
    auto store_state = [&](float *dst) {
        scale_state(fast_exp2(static_cast<float>(level)));
        level = 0.0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) v[ct] = S[nt][ct][r];
                lanevec<float, CT>::st(lane_at(dst + (16 * nt + r) * p.P, 4 * g * p.P + c16 * CT), v);
            }
    };

    // zero what no staging writes: columns past d_state, the score tiles above the diagonal
    if (NS < 32)
        for (int b = 0; b < NBUF; ++b)
            for (int i = tid; i < Cf::BN + (FULL ? Cf::CN : 0); i += 64 * NW) Bn(b, 0)[i] = 0;
    if (FULL)
        for (int b = 0; b < NBUF; ++b)
            for (int i = tid; i < Cf::GT; i += 64 * NW) Gt(b, 0)[i] = 0;
    if (FULL || NS < 32) lds_barrier();

    // Staging of a chunk's B and C: a thread takes 4 tokens by 4 channels.
    // Rows past the segment repeat its last one: their step size is 0, so
    // whatever they hold meets a factor of 0 or a row that is not stored.  Rows
    // are clamped rather than branched on: a wait behind a branch counts no
    // request made inside.
    constexpr int BLOCKS = (L / 4) * (NS / 4), PER = (BLOCKS + 64 * NW - 1) / (64 * NW);
    constexpr int AHEAD = FULL ? 1 : 2;  // chunks between a request and its use: the states alone are a short iteration
    quad<TI> rawB[AHEAD][PER], rawC[FULL ? PER : 1];
    auto fetch = [&](int c, quad<TI> (&raw)[PER]) {
        const int rem = min(sg.len - c * L, L);
        const TI *b0 = bb + static_cast<int64_t>(c) * L * p.b_st, *c0 = cb + static_cast<int64_t>(c) * L * p.c_st;
        const uint32_t bs = static_cast<uint32_t>(p.b_st), cs = static_cast<uint32_t>(p.c_st);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t i = min(tid + k * 64 * NW, BLOCKS - 1);  // the threads to spare repeat the last block
            const uint32_t t = 4 * (i / (NS / 4)), n = 4 * (i % (NS / 4)), bt = t * bs, ct = t * cs;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                raw[k].ld(r, lane_at(b0, min(bt + r * bs, (rem - 1) * bs) + n));
                if constexpr (FULL) rawC[k].ld(r, lane_at(c0, min(ct + r * cs, (rem - 1) * cs) + n));
            }
        }
    };
    auto stage = [&](int b, const quad<TI> (&raw)[PER]) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid + k * 64 * NW;
            const int tq = i / (NS / 4), nq = i % (NS / 4);
            if (BLOCKS % (64 * NW) == 0 || i < BLOCKS)
#pragma unroll
                for (int part = 0; part < EX; ++part)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        *reinterpret_cast<uint2 *>(Bn(b, part) + (tq * 4 + r) * RB + col_pos(nq * 4)) = raw[k].row(r, part).u;
                        if (FULL) *reinterpret_cast<uint2 *>(Cn(b, part) + (tq * 4 + r) * RN + col_pos(nq * 4)) = rawC[k].row(r, part).u;
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
                    load_rows(a.f[part], Bn(b, part), RB, 16 * tj, kk, g, c16);
                    load_rows(bf.f[part], Cn(b, part), RN, 16 * ti, kk, g, c16);
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
    // x (rows in the operand's slot order) and dt of a chunk; a lane's token is
    // its own number in the reverse mode (sums from the chunk's start are
    // wanted), else counted from the chunk's end
    lanevec<TI, CT> xs[AHEAD][TK][8];
    typedef typename std::conditional<Cf::BF, uint32_t, float>::type Step;
    float dt_next;  // of the chunk to come
    auto token = [&] { return REV ? tid & 63 : L - 1 - (tid & 63); };
    auto fetch_dt = [&](int c, Step &d) {
        const int rem = min(sg.len - c * L, L);
        d = *lane_at(dtb + static_cast<int64_t>(c) * L * p.H, max(0, min(token(), rem - 1)) * p.H);
    };
    // The step sizes requested at a chunk's start are taken up at its end: a
    // 16-bit value carried into the next iteration would be widened, and waited
    // for, wherever the compiler likes.
    auto take_dt = [&](Step &d) {
        asm volatile("" : "+v"(d));
        if constexpr (Cf::BF) dt_next = __uint_as_float(d << 16);
        else dt_next = d;
    };
    auto fetch_x = [&](int c, lanevec<TI, CT> (&xv)[TK][8]) {
        const int rem = min(sg.len - c * L, L);
        const TI *base = xb + static_cast<int64_t>(c) * L * p.x_st;
        const uint32_t row = 4 * g * x_st, last = (rem - 1) * x_st;
#pragma unroll
        for (int ks = 0; ks < TK; ++ks)
#pragma unroll
            for (int j = 0; j < 8; ++j) xv[ks][j].ld(lane_at(base, min(row + (32 * ks + kperm(0, j)) * x_st, last) + c16 * CT));
    };

    const int chunks = __builtin_amdgcn_readfirstlane((sg.len + L - 1) / L);
    float seg_log = 0.f;
    // the i-th chunk of the walk; past the end the last one again: requests are
    // made on every path, so that a wait can count those made after it
    auto order = [&](int i) { return REV ? max(chunks - 1 - i, 0) : min(i, chunks - 1); };
    // the shared part of a chunk's step, before and after a wave's own: all
    // waves stage B and C and take a part of the scores
    auto request = [&](int i, quad<TI> (&raw)[PER]) {
        // what follows from the lane's place is computed again in every
        // iteration: kept over the loop it would push the tiles out of the
        // registers, and every spill waits for all loads in flight
        asm volatile("" : "+v"(g), "+v"(c16), "+v"(tid));
        if (NBUF == 2) {  // the next chunk into the other buffer
            stage((i & 1) ^ 1, raw);
            fetch(order(i + 1 + AHEAD), raw);
        }
    };
    auto score = [&](int i) {
        if (FULL && NBUF == 2) {  // the next chunk is staged: its scores, beside this chunk's products
            lds_barrier();
            if (i + 1 < chunks) scores((i & 1) ^ 1);
        }
    };
    auto finish = [&](int i, quad<TI> (&raw)[PER]) {
        lds_barrier();
        if (NBUF == 1 && i + 1 < chunks) {
            stage(0, raw);
            fetch(order(i + 1 + AHEAD), raw);
            lds_barrier();
            if (FULL) {
                scores(0);
                lds_barrier();
            }
        }
    };
    // Whole chunks (WHOLE) take no branch around a store: behind one, a wait for
    // an older load would have to count on the stores not having been made, and
    // so wait for them too.
    auto body = [&](auto whole, int i, lanevec<TI, CT> (&xr)[TK][8], quad<TI> (&raw)[PER]) {
        constexpr bool WHOLE = decltype(whole)::value;
        const int b = NBUF == 2 ? i & 1 : 0;
        const int t0 = order(i) * L, rem = WHOLE ? L : i < chunks ? min(sg.len - t0, L) : 0;
        Step d;
        fetch_dt(order(i + 1), d);
        request(i, raw);
        float dec = 1.f;
        bool fast = true, late = false;
        f32x4 acc[FULL ? ST : 1][CT];
        {
            // the state entering the chunk (from the right in the reverse order)
            if (phase == 2 && p.chunk_states && i < chunks && t0 % q.state_chunk == 0)
                store_state(p.chunk_states + ((static_cast<int64_t>(sg.chunk + t0 / 64) * (64 / q.state_chunk) + t0 % 64 / q.state_chunk) * p.H + h) * per_head + pw0);
            // decays, one token a lane
            const int tok = token(), lane = tid & 63;
            float dt = dt_next + bias;
            if (p.softplus) dt = softplus_rel(dt);
            if (tok < 0 || tok >= rem) dt = 0.f;
            float la = A2 * dt;
            if (la < kGone) la = kGone;
            // from the chunk's end (reverse: its start) to the token.  The states
            // alone take no difference of two sums: a sum large enough to be coarse
            // has left nothing
            typedef typename std::conditional<FULL, double, float>::type Sum;
            const Sum incl = lane_scan(static_cast<Sum>(la));
            const Sum tot = last_lane(incl);
            fast = !FULL || fabs(tot) < kFastTot;
            const float from = static_cast<float>(level);
            double next = level + tot;
            const bool wide = FULL && fast && fabs(tot) > kFastTot / 2;
            const bool out = __builtin_amdgcn_readfirstlane(wide || !(fabs(next) <= kLevel));
            const double to = wide ? 0.5 * tot : 0.0;
            dec = fast_exp2(static_cast<float>(next - to));
            if (out) next = to;
            level = next;
            if (fast && out) scale_state(dec);  // the second form reads the state before this chunk's decay
            const float hi = static_cast<float>(next), lo = static_cast<float>(next - hi);
            if (REV) {
                if (lane < L) wv[lane] = lane < rem ? fast_exp2((incl - hi) - lo) : 0.f;
            } else {
                const Sum suf = lane_shift(incl);
                if (tok >= 0) {
                    if constexpr (FULL) {
                        wv[tok] = dt * fast_exp2(static_cast<float>(suf - next));
                        fv[tok] = fast ? fast_exp2(static_cast<float>(next - suf)) : la;
                        sv[tok] = static_cast<float>(suf);
                        sl[tok] = static_cast<float>(suf - static_cast<float>(suf));
                        dv[tok] = dt;
                    } else {
                        wv[tok] = dt * fast_exp2((suf - hi) - lo);
                    }
                }
                if (FULL && !fast) {  // the sums from the chunk's start
                    wave_lds_fence();
                    const float cum = lane_scan(lane < L ? fv[lane] : 0.f);
                    wave_lds_fence();
                    if (lane < L) fv[lane] = fast_exp2(cum + from);
                }
            }
            seg_log += static_cast<float>(tot);
            late = !fast && out;
            wave_lds_fence();
            if constexpr (FULL) {  // C S
#pragma unroll
                for (int s = 0; s < ST; ++s)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) acc[s][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    parts8<SP> sf[CT];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int r = 0; r < 4; r += 2) {
                            constexpr f32x4 none = {0.f, 0.f, 0.f, 0.f};
                            const f32x4 &s1 = 2 * kk + 1 < NT ? S[2 * kk + 1 < NT ? 2 * kk + 1 : 0][ct] : none;
                            split_pair<SP>(sf[ct], r, S[2 * kk][ct][r], S[2 * kk][ct][r + 1]);
                            split_pair<SP>(sf[ct], 4 + r, s1[r], s1[r + 1]);
                        }
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        parts8<EX> a;
#pragma unroll
                        for (int part = 0; part < EX; ++part) load_rows(a.f[part], Cn(b, part), RN, 16 * s, kk, g, c16);
                        mfma_tiles<EX, SP, ORD, CT>(acc[s], a, sf);
                    }
                }
                if (!fast)
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        const f32x4 f = *reinterpret_cast<const f32x4 *>(fv + 16 * s + 4 * g);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) acc[s][ct] *= f;
                    }
                if (late) scale_state(dec);
            }
        }
        score(i);
        {
            if constexpr (FULL) {
                if (!fast) {  // the second form's intra-chunk part
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        const int row = 16 * s + c16;
                        const float suf_row = sv[row], low_row = sl[row];
#pragma unroll
                        for (int ks = 0; ks <= s / 2; ++ks) {
                            asm volatile("" ::: "memory");  // the factors are read again, not kept over the strips
                            __builtin_amdgcn_sched_barrier(0);
                            parts8<GP> m;
#pragma unroll
                            for (int part = 0; part < GP; ++part) load_rows(m.f[part], Gt(b, part), RT, 16 * s, ks, g, c16);
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
                                const f32x4 lc = *reinterpret_cast<const f32x4 *>(sl + col);
                                const f32x4 dc = *reinterpret_cast<const f32x4 *>(dv + col);
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const float k = col + r <= row ? dc[r] * fast_exp2((sc[r] - suf_row) + (lc[r] - low_row)) : 0.f;
                                    split_to<GP>(m, 4 * hq + r, mv[4 * hq + r] * k);
                                }
                            }
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) {
                                parts8<EX> xe;
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    lanevec<TI, CT> v = xr[ks][j];
                                    asm volatile("" : "+v"(v.u));
                                    split_to<EX>(xe, j, v.get(ct));
                                }
                                mfma_parts<GP, EX, ORD>(acc[s][ct], m, xe);
                            }
                        }
                    }
                }
            }
            // w x, 32 tokens at a time: into y through the scores, into S through B
#pragma unroll
            for (int ks = 0; ks < TK; ++ks) {
                parts8<XP> xw[CT];
#pragma unroll
                for (int hq = 0; hq < 2; ++hq) {
                    const f32x4 wq = *reinterpret_cast<const f32x4 *>(wv + 32 * ks + 16 * hq + 4 * g);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int r = 0; r < 4; r += 2)
                            split_pair<XP>(xw[ct], 4 * hq + r, xr[ks][4 * hq + r].get(ct) * wq[r], xr[ks][4 * hq + r + 1].get(ct) * wq[r + 1]);
                }
                if constexpr (FULL) {
                    if (fast)
#pragma unroll
                        for (int s = 2 * ks; s < ST; ++s) {
                            parts8<GP> a;
#pragma unroll
                            for (int part = 0; part < GP; ++part) load_rows(a.f[part], Gt(b, part), RT, 16 * s, ks, g, c16);
                            mfma_tiles<GP, XP, ORD, CT>(acc[s], a, xw);
                        }
                }
                // several tiles' operands requested together, and their products
                // taken part by part: no instruction waits for the one before
                constexpr int NG = EX == 1 ? (NT < 8 ? NT : 8) : 1;
#pragma unroll
                for (int n0 = 0; n0 < NT; n0 += NG) {
                    parts8<EX> a[NG];
#pragma unroll
                    for (int k = 0; k < NG; ++k)
#pragma unroll
                        for (int part = 0; part < EX; ++part) load_cols(a[k].f[part], Bn(b, part), RB, 32 * ks, 16 * (n0 + k), g, c16);
#pragma unroll
                    for (int i0 = 0; i0 < EX; ++i0)
#pragma unroll
                        for (int j0 = 0; i0 + j0 < 3 && j0 < XP; ++j0)
#pragma unroll
                            for (int k = 0; k < NG; ++k)
#pragma unroll
                                for (int ct = 0; ct < CT; ++ct) S[n0 + k][ct] = mfma16(a[k].f[i0].v, xw[ct].f[j0].v, S[n0 + k][ct]);
                }
            }
            if constexpr (FULL) {  // y: slot (s % 2) 4 + r of x's step s / 2 is the same row
                TO *yc = yb + static_cast<int64_t>(t0) * y_st;
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    f32x4 f = {1.f, 1.f, 1.f, 1.f};
                    if (fast) f = *reinterpret_cast<const f32x4 *>(fv + 16 * s + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float v[CT];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) v[ct] = fmaf(Dh, xr[s / 2][(s % 2) * 4 + r].get(ct), acc[s][ct][r] * f[r]);
                        if (WHOLE || 16 * s + 4 * g + r < rem)
                            lanevec<TO, CT>::st(lane_at(yc + (16 * s + r) * static_cast<int64_t>(y_st), 4 * g * y_st + c16 * CT), v);
                    }
                }
            }
        }
        take_dt(d);
        fetch_x(order(i + AHEAD), xr);
        finish(i, raw);
    };
    if (chunks > 0) {
        fetch(order(0), rawB[0]);
        Step d;
        fetch_dt(order(0), d);
        take_dt(d);
        fetch_x(order(0), xs[0]);
        stage(0, rawB[0]);
        // chunk c's B and C wait in set c % AHEAD
        fetch(order(1), rawB[1 % AHEAD]);
        if (AHEAD == 2) fetch_x(order(1), xs[AHEAD - 1]);
        if (AHEAD == 2) fetch(order(2), rawB[0]);
        lds_barrier();
        if (FULL) {
            scores(0);
            lds_barrier();
        }
    }
    // nothing is in flight where the loops are entered: their waits count from
    // the worst of all the ways in
    auto settle = [] {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
    };
    settle();
    if (!on) {  // as many barriers as the others
        auto step = [&](int i, quad<TI> (&raw)[PER]) {
            request(i, raw);
            score(i);
            finish(i, raw);
        };
        for (int i = 0; i < chunks; i += AHEAD) {
            step(i, rawB[AHEAD - 1]);
            if (AHEAD == 2) step(i + 1, rawB[0]);
        }
        settle();
        return;
    }
    int i = 0;
    if constexpr (FULL) {
        for (const int whole = sg.len / L; i < whole; ++i) body(std::true_type{}, i, xs[0], rawB[0]);
        if (i < chunks) body(std::false_type{}, i, xs[0], rawB[0]);
    } else {
        // two at a time, with no exit between them that a wait would have to
        // allow for; an odd last chunk is followed by one of no tokens
        for (; i < chunks; i += 2) {
            body(std::false_type{}, i, xs[0], rawB[AHEAD - 1]);
            body(std::false_type{}, i + 1, xs[AHEAD - 1], rawB[0]);
        }
    }
    if (phase == 1) {
        store_state(q.seg_state + (static_cast<int64_t>(x_seg) * p.H + h) * per_head + pw0);
        if (pc == 0 && g == 0) q.seg_log[static_cast<int64_t>(x_seg) * p.H + h] = seg_log;
    } else if (p.final_state && (REV ? sg.s == 0 : sg.s == sg.count - 1)) {
        store_state(p.final_state + (static_cast<int64_t>(sg.n) * p.H + h) * per_head + pw0);
    }
}

// at most two waves a SIMD (the LDS holds one workgroup): all registers of two
template <typename TI, typename TO, int NS, int PW, int NW, int MODE>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4)))
ssm_scan_kernel(SsmScan q, int blocks_per_group, int phase) {
    __shared__ __attribute__((aligned(16))) char smem[ScanCfg<TI, TO, NS, PW, NW, MODE>::BYTES];
    ssm_scan<TI, TO, NS, PW, NW, MODE>(smem, q, blockIdx.x, gridDim.x, blocks_per_group, phase);
}
// the states from the left, and with the second half of the grid from the right
template <typename TI, int NS, int PW, int NW>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4)))
ssm_states_kernel(SsmScan f, SsmScan r, int blocks_per_group, int phase) {
    __shared__ __attribute__((aligned(16))) char smem[ScanCfg<TI, float, NS, PW, NW, SSM_STATES>::BYTES];
    const int half = gridDim.x / 2;
    if (blockIdx.x < half) ssm_scan<TI, float, NS, PW, NW, SSM_STATES>(smem, f, blockIdx.x, half, blocks_per_group, phase);
    else ssm_scan<TI, float, NS, PW, NW, SSM_REVERSE>(smem, r, blockIdx.x - half, half, blocks_per_group, phase);
}

inline unsigned scan_grid(const SsmScan &q, const SsmPlan &plan) {
    const int64_t want = static_cast<int64_t>(plan.segs_bound) * q.p.G * plan.blocks_per_group;
    return static_cast<unsigned>((want + 7) / 8 * 8);
}
template <typename TI, typename TO, int NS, int PW, int MODE>
hipError_t run(const SsmScan &q, const SsmPlan &plan, int phase, hipStream_t s) {
    const unsigned grid = scan_grid(q, plan);
    if (plan.waves == 8)
        hipLaunchKernelGGL((ssm_scan_kernel<TI, TO, NS, PW, 8, MODE>), dim3(grid), dim3(512), 0, s, q, plan.blocks_per_group, phase);
    else
        hipLaunchKernelGGL((ssm_scan_kernel<TI, TO, NS, PW, 4, MODE>), dim3(grid), dim3(256), 0, s, q, plan.blocks_per_group, phase);
    return hipGetLastError();
}
template <typename TI, int NS, int PW>
hipError_t run_states(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int phase, hipStream_t s) {
    const unsigned grid = 2 * scan_grid(f, plan);
    if (plan.waves == 8)
        hipLaunchKernelGGL((ssm_states_kernel<TI, NS, PW, 8>), dim3(grid), dim3(512), 0, s, f, r, plan.blocks_per_group, phase);
    else
        hipLaunchKernelGGL((ssm_states_kernel<TI, NS, PW, 4>), dim3(grid), dim3(256), 0, s, f, r, plan.blocks_per_group, phase);
    return hipGetLastError();
}
template <typename TI, typename TO, int NS>
hipError_t run_p(const SsmScan &q, const SsmPlan &plan, int phase, hipStream_t s) {
    if (q.p.P == 16)
        return phase == 2 ? run<TI, TO, NS, 16, SSM_FULL>(q, plan, phase, s) : run<TI, float, NS, 16, SSM_STATES>(q, plan, phase, s);
    return phase == 2 ? run<TI, TO, NS, 32, SSM_FULL>(q, plan, phase, s) : run<TI, float, NS, 32, SSM_STATES>(q, plan, phase, s);
}
template <typename TI, int NS>
hipError_t run_states_p(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int phase, hipStream_t s) {
    return f.p.P == 16 ? run_states<TI, NS, 16>(f, r, plan, phase, s) : run_states<TI, NS, 32>(f, r, plan, phase, s);
}
}  // namespace

template <typename TI, typename TO>
hipError_t ssm_phase(const SsmScan &q, const SsmPlan &plan, int phase, hipStream_t s) {
    switch (q.p.Ns) {
        case 16: return run_p<TI, TO, 16>(q, plan, phase, s);
        case 32: return run_p<TI, TO, 32>(q, plan, phase, s);
        case 64: return run_p<TI, TO, 64>(q, plan, phase, s);
        default: return run_p<TI, TO, 128>(q, plan, phase, s);
    }
}
template <typename TI>
hipError_t ssm_states(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int phase, hipStream_t s) {
    switch (f.p.Ns) {
        case 16: return run_states_p<TI, 16>(f, r, plan, phase, s);
        case 32: return run_states_p<TI, 32>(f, r, plan, phase, s);
        case 64: return run_states_p<TI, 64>(f, r, plan, phase, s);
        default: return run_states_p<TI, 128>(f, r, plan, phase, s);
    }
}

}  // namespace kda
