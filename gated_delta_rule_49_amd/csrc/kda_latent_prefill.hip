// Latent attention's expanded form on the bf16 matrix cores: the forward.
//
// A workgroup of four waves takes 128 queries of one head, a wave 32 of them, and
// walks the keys 64 at a time.  S^T = K Q^T, so that a lane holds 32 scores of ONE
// query (its partner in the other half the other 32): the softmax needs one
// exchange for the maximum, and P goes on to O^T += V^T P^T in its registers.
// Keys and values come from memory to LDS directly, one tile ahead in the other
// buffer, with one barrier a tile; two workgroups of a CU (80 KB of LDS and up to
// 256 registers a wave each) let one's softmax run under the other's products.
//
// Softmax: the running maximum moves only when a score passes it by more than
// kSlack (log2), which few tiles do after the first; until then P may be as large
// as 2^kSlack, which costs a bf16 or an fp32 sum nothing.
//
// P enters the second product as one bf16 operand, which rounds each term of a sum
// by up to 2^-8 of itself, or, where the caller asks for it (precise), as two, which
// round by 2^-16.  Both sides, 8192 tokens as below: 678 us for 897; the error of a
// bf16 o against 64 bits 2.1e-3 for 1.6e-3, of which its own rounding is 1.6e-3.
//
// 8192 tokens of 32 heads (keys 192, values 128, causal): 667 us, 1.03 PFLOP/s.
// Matrix instructions take 54 % of the cycles and vector ones (the softmax) 55 %,
// at the 1.7 GHz that this load leaves; LDS 27 %, without bank conflicts.
#include "kda_latent_bf16.hpp"

namespace kda {

namespace {

constexpr int kTileQ = 128, kKeys = 64, kThreads = 256;
constexpr float kSlack = 8.f;

template <typename O, int DK, int DV, int PARTS>
__global__ void __launch_bounds__(kThreads, 2) prefill_bf16_kernel(LatentParams p) {
    constexpr int KB = kKeys * DK * 2, VB = kKeys * DV * 2;
    __shared__ __attribute__((aligned(16))) char s_tile[2 * (KB + VB)];
    const LatentPlace a = latent_place(p, p.tq, blockIdx.x, p.causal);
    if (!a.valid) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, c32 = lane & 31;
    const bf16_t *kn = static_cast<const bf16_t *>(p.kn) + a.b * p.k_sb + a.h * p.k_sh + a.k0 * p.k_st;
    const bf16_t *kr = static_cast<const bf16_t *>(p.kr) + a.b * p.r_sb + a.k0 * p.r_st;
    const bf16_t *v = static_cast<const bf16_t *>(p.v) + a.b * p.v_sb + a.h * p.v_sh + a.k0 * p.v_st;
    const int q_first = a.tile * kTileQ + wave * 32, qi = q_first + c32;
    const int shift = a.tk - a.tq;
    const int n = p.causal ? min(a.tk, min(a.tq, (a.tile + 1) * kTileQ) + shift) : a.tk;
    // keys that the wave's queries see: the first one's, the last one's, the lane's
    const int n_least = p.causal ? min(n, q_first + shift + 1) : n;
    const int n_wave = q_first >= a.tq ? 0 : p.causal ? min(n, min(a.tq - 1, q_first + 31) + shift + 1) : n;
    const int limit = p.causal ? min(n, qi + shift + 1) : n;

    TileLoader<DK, kKeys, kThreads, RowRead, true> keys;
    TileLoader<DV, kKeys, kThreads, ColumnRead, false> values;
    keys.init(kn, p.k_st, p.dn, kr, p.r_st, p.dr, 0);
    values.init(v, p.v_st, p.dv, v, 0, 0, 0);
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_address(s_tile));
    if (n > 0) {
        keys.issue(0, n, lds);
        values.issue(0, n, lds + 2 * KB);
    }
    bf16x8 qf[DK / 16];
    load_own<DK>(qf, static_cast<const bf16_t *>(p.q) + a.b * p.q_sb + a.h * p.q_sh + (static_cast<int64_t>(a.q0) + min(qi, a.tq - 1)) * p.q_st, p.dn + p.dr, kr, 0,
                 qi < a.tq && p.scale != 0.f, h);
    if (p.scale < 0.f) {  // scores are masked before they are scaled: the scale's sign goes to the query
#pragma unroll
        for (int s = 0; s < DK / 16; ++s) {
            frag8 f;
            f.v = qf[s];
            f.u = make_uint4(f.u.x ^ 0x80008000u, f.u.y ^ 0x80008000u, f.u.z ^ 0x80008000u, f.u.w ^ 0x80008000u);
            qf[s] = f.v;
        }
    }
    const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e;
    f32x16 acc[DV / 32];
#pragma unroll
    for (int b = 0; b < DV / 32; ++b) acc[b] = zero16();
    float top = -INFINITY, sum = 0.f;
    // the lane's places in a tile: its key's row; four rows by 16 channels
    const int i16 = lane & 15, g2 = (lane >> 4) & 1;
    const char *v_at = s_tile + 2 * KB + (4 * h + (i16 >> 2)) * DV * 2 + 8 * (i16 & 1);

    for (int k0 = 0, buf = 0; k0 < n; k0 += kKeys, buf ^= 1) {
        wait_loads();
        lds_barrier();
        if (k0 + kKeys < n) {
            keys.issue(k0 + kKeys, n, lds + (buf ^ 1) * KB);
            values.issue(k0 + kKeys, n, lds + 2 * KB + (buf ^ 1) * VB);
        }
        if (k0 >= n_wave) continue;
        __builtin_amdgcn_s_setprio(1);
        f32x16 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = zero16();
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                frag8 f;
                f.u = *reinterpret_cast<const uint4 *>(s_tile + buf * KB + 32 * t * DK * 2 + RowRead::place<DK>(c32, 2 * k + h));
                s[t] = mfma32(f.v, qf[k], s[t]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        if (k0 + kKeys > n_least) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3) >= limit) s[t][i] = -INFINITY;
        }
        float m2[2] = {s[0][0], s[1][0]};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 1; i < 15; i += 2) m2[t] = fmaxf(fmaxf(s[t][i], s[t][i + 1]), m2[t]);
        const float most = swap_halves_max(fmaxf(fmaxf(m2[0], s[0][15]), fmaxf(m2[1], s[1][15]))) * c;
        if (__any(most > top + kSlack)) {
            const float next = fmaxf(top, most);
            const float keep = next == -INFINITY ? 1.f : fast_exp2(top - next);
            top = next;
            sum *= keep;
#pragma unroll
            for (int b = 0; b < DV / 32; ++b) acc[b] *= keep;
        }
        const float base = top == -INFINITY ? 0.f : top;
        bf16x8 pf[4][PARTS];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = fast_exp2(fmaf(s[t][i], c, -base));
            }
            sum += ((s[t][0] + s[t][1]) + (s[t][2] + s[t][3]) + ((s[t][4] + s[t][5]) + (s[t][6] + s[t][7]))) + (((s[t][8] + s[t][9]) + (s[t][10] + s[t][11])) + ((s[t][12] + s[t][13]) + (s[t][14] + s[t][15])));
            half_tile(pf[2 * t], s[t], 0);
            half_tile(pf[2 * t + 1], s[t], 1);
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int b = 0; b < DV / 32; ++b) {
            const int chunk = 4 * b + 2 * g2 + ((i16 & 3) >> 1);
            const char *at = v_at + buf * VB + (ColumnRead::place<DV>(i16 >> 2, chunk) - (i16 >> 2) * DV * 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint2 lo = read_tr16(at + 16 * k * DV * 2), hi = read_tr16(at + (16 * k + 8) * DV * 2);
                frag8 f;
                f.u = make_uint4(lo.x, lo.y, hi.x, hi.y);
                acc[b] = mfma32(f.v, pf[k], acc[b]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
    }
    sum = swap_halves_sum(sum);
    if (qi >= a.tq) return;
    const int64_t row = (a.q_row + qi) * p.H + a.h;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    O *o = static_cast<O *>(p.o) + row * p.dv;
#pragma unroll
    for (int b = 0; b < DV / 32; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = 32 * b + 8 * i + 4 * h;
            if (ch >= p.dv) continue;
            store4(o + ch, acc[b], i, inv);
        }
    if (h == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <typename O, int DK, int DV>
hipError_t run(const LatentParams &p, hipStream_t s) {
    const int grid = p.cu_q ? p.H * p.tq.bound : p.H * p.N * p.tq.per_seq;
    if (p.precise) prefill_bf16_kernel<O, DK, DV, 2><<<grid, kThreads, 0, s>>>(p);
    else prefill_bf16_kernel<O, DK, DV, 1><<<grid, kThreads, 0, s>>>(p);
    return hipGetLastError();
}
template <typename O>
hipError_t pick(const LatentParams &p, hipStream_t s) {
    const int dk = p.dn + p.dr;
    if (dk <= 64 && p.dv <= 64) return run<O, 64, 64>(p, s);
    if (dk <= 128) return run<O, 128, 128>(p, s);
    return run<O, 192, 128>(p, s);
}

}  // namespace

int latent_tile_q(int dtype, int64_t tokens, int H) { return dtype == 0 ? latent_tile_f32(tokens, H) : kTileQ; }

hipError_t launch_latent_prefill(const LatentParams &p, int in_dtype, int out_dtype, hipStream_t s) {
    if (in_dtype == 0) return latent_prefill_f32(p, out_dtype, s);
    return out_dtype == 0 ? pick<float>(p, s) : pick<bf16_t>(p, s);
}

}  // namespace kda
