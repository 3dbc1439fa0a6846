// The stages after a block and before the next one in one pass over the rows:
// norm of the block's output, gate, scaled residual, norm of the sum (the
// "gated norm" and residual stages of the executed sublayer, Module 04 —
// KDA II, §3 "The sublayer is bigger than the recurrence"), and the gradients.
//
// Per row, q = 1 / sqrt(mean_group(a^2) + eps), q2 = 1 / sqrt(mean(out^2) + eps):
//     a = x (or x act(z), gate first),  v = a q w (times act(z), gate after)
//     out = r + s v,                    normed = out q2 w2
// and backwards, with do, dn the gradients of out and normed:
//     e2 = dn w2,   dO = do + q2 e2 - out q2^3 mean(e2 out)
//     dr = dO,  ds += dO v,  dw2 += dn out q2
//     dv = dO s,  (gate after: dz = dv a q w act'(z), dv = dv act(z))
//     dw += dv a q,  e = dv w,  da = q e - a q^3 mean_group(e a)
//     dx = da (gate first: dz = da x act'(z), dx = da act(z))
//
// HBM-bound: every plane is read once and written once; all sums in fp32.
// A team of TS threads (one wave to a whole workgroup) owns a row and keeps
// it in registers, CPT vectors of VEC channels a thread, so the reductions
// cost no second read.  Teams walk the rows with a grid stride: the weights
// stay in registers, and the next row's vectors are requested before this
// row's reductions wait.
//
// 8192 rows of 4096 bf16 channels, residual, scale and both norms: forward
// 61 us (4.4 TB/s; a copy of the same bytes takes 52), gradients 131 us (a copy:
// 104), of which 5 are the column sums of the three weights' partial rows.
//
// Wider rows: from 4097 channels on 1024 threads hold 8 channels each in the
// gradients, from 8193 on 16 (and 16 in the forward), which spill.  2^25 bf16
// channels, residual, scale and both norms: forward 62, 74, 67, 254 us for rows of
// 4096, 5120, 8192, 16384 (a copy 52), gradients 144, 632, 525, 1016 (a copy 78).
#include "kda_launch.hpp"

namespace kda {

namespace {

template <typename T, int VEC> struct rowvec;
template <> struct rowvec<bf16_t, 8> {
    uint4 u;
    __device__ void ld(const bf16_t *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ float get(int c) const {
        const uint32_t w = c < 2 ? u.x : c < 4 ? u.y : c < 6 ? u.z : u.w;
        return __uint_as_float((c & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ static void st(bf16_t *p, const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = static_cast<uint32_t>(f32_to_bf16(v[2 * i])) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct rowvec<float, 8> {
    float4 a, b;
    __device__ void ld(const float *p) { a = reinterpret_cast<const float4 *>(p)[0]; b = reinterpret_cast<const float4 *>(p)[1]; }
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ float get(int c) const {
        const float4 &h = c < 4 ? a : b;
        const int k = c & 3;
        return k == 0 ? h.x : k == 1 ? h.y : k == 2 ? h.z : h.w;
    }
    __device__ static void st(float *p, const float (&v)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <> struct rowvec<bf16_t, 4> {
    uint2 u;
    __device__ void ld(const bf16_t *p) { u = *reinterpret_cast<const uint2 *>(p); }
    __device__ void zero() { u = make_uint2(0, 0); }
    __device__ float get(int c) const {
        const uint32_t w = c < 2 ? u.x : u.y;
        return __uint_as_float((c & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ static void st(bf16_t *p, const float (&v)[4]) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(
            static_cast<uint32_t>(f32_to_bf16(v[0])) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
            static_cast<uint32_t>(f32_to_bf16(v[2])) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
    }
};
template <> struct rowvec<float, 4> {
    float4 u;
    __device__ void ld(const float *p) { u = *reinterpret_cast<const float4 *>(p); }
    __device__ void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ float get(int c) const { return c == 0 ? u.x : c == 1 ? u.y : c == 2 ? u.z : u.w; }
    __device__ static void st(float *p, const float (&v)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
};
template <typename T> struct rowvec<T, 1> {
    T u;
    __device__ void ld(const T *p) { u = *p; }
    __device__ void zero() { u = T(0); }
    __device__ float get(int) const { return io<T>::ld(&u, 0); }
    __device__ static void st(T *p, const float (&v)[1]) { io<T>::st(p, 0, v[0]); }
};

// 1 / (1 + e^-z) with the hardware's reciprocal (1 ulp); e^-z overflows to
// infinity where the result is 0
__device__ __forceinline__ float gate_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e)); }
// the gate's activation and its derivative
__device__ __forceinline__ float gate_act(float z, int silu) {
    const float s = gate_sigmoid(z);
    return silu ? z * s : s;
}
__device__ __forceinline__ void gate_act_grad(float z, int silu, float &act, float &slope) {
    const float s = gate_sigmoid(z);
    act = silu ? z * s : s;
    slope = silu ? fmaf(z * s, 1.f - s, s) : s * (1.f - s);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// Sums over a team of TS threads; `slot` [TS / 64] floats of LDS of its own
// for each call between two uses.
template <int TS>
__device__ __forceinline__ float team_sum(float v, float *slot, int tid) {
    v = wave_sum(v);
    if (TS > 64) {
        if ((tid & 63) == 0) slot[tid >> 6] = v;
        lds_barrier();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TS / 64; ++w) v += slot[w];
    }
    return v;
}

// How group sums are taken: over the team (group == dim), over 2^k lanes of a
// wave, or through LDS (any other group).
enum { GROUP_ROW = 0, GROUP_LANES = 1, GROUP_LDS = 2 };

// The sums over each channel's group of val[j][c].  Where a group is a row or
// 2^k lanes, a thread's vector lies in one group and has one sum.  LDS: every
// channel's value goes through LDS `buf` [dim], the waves of the team sum the
// groups into `sums` [dim / group], and each channel looks its own up.
template <int VEC, int CPT, int TS, bool LDS>
__device__ __forceinline__ void group_sums(const float (&val)[CPT][VEC], float (&sum)[CPT][LDS ? VEC : 1], const NormParams &p, int mode,
                                           float *slot, float *buf, int tid) {
    if constexpr (!LDS) {
        float part[CPT];
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            part[j] = 0.f;
#pragma unroll
            for (int c = 0; c < VEC; ++c) part[j] += val[j][c];
        }
        if (mode == GROUP_ROW) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < CPT; ++j) s += part[j];
            s = team_sum<TS>(s, slot, tid);
#pragma unroll
            for (int j = 0; j < CPT; ++j) sum[j][0] = s;
        } else {
            const int lanes = p.group / VEC;
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                for (int m = 1; m < lanes; m <<= 1) part[j] += __shfl_xor(part[j], m);
                sum[j][0] = part[j];
            }
        }
    } else {
        float *sums = buf + p.dim;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int e0 = (tid + j * TS) * VEC;
            if (e0 < p.dim)
#pragma unroll
                for (int c = 0; c < VEC; ++c) buf[e0 + c] = val[j][c];
        }
        lds_barrier();
        const int ng = p.dim / p.group;
        for (int g = tid >> 6; g < ng; g += TS / 64) {
            float s = 0.f;
            for (int e = tid & 63; e < p.group; e += 64) s += buf[g * p.group + e];
            s = wave_sum(s);
            if ((tid & 63) == 0) sums[g] = s;
        }
        lds_barrier();
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int e0 = (tid + j * TS) * VEC;
            if (e0 < p.dim)
#pragma unroll
                for (int c = 0; c < VEC; ++c) sum[j][c] = sums[(e0 + c) / p.group];
        }
        lds_barrier();  // buf is free again
    }
    // channels past the row hold zeros; their mean stays one, so that no
    // 0 / 0 of theirs reaches the row's sums (eps may be 0)
#pragma unroll
    for (int j = 0; j < CPT; ++j)
        if ((tid + j * TS) * VEC >= p.dim)
#pragma unroll
            for (int c = 0; c < (LDS ? VEC : 1); ++c) sum[j][c] = 1.f;
}

// LDS floats one team needs
__host__ __device__ inline int team_lds_floats(int ts, bool buf, int dim, int group) {
    return 3 * (ts / 64) + (buf ? dim + dim / group : 0);
}

template <typename T, int VEC, int CPT, int TS>
struct RowBuf {  // one row's inputs as loaded
    rowvec<T, VEC> x[CPT], z[CPT], r[CPT];
    __device__ __forceinline__ void load(const NormParams &p, int64_t row, int tid) {
        const T *px = static_cast<const T *>(p.x) + row * p.x_stride;
        const T *pz = static_cast<const T *>(p.gate) + row * p.gate_stride;
        const T *pr = static_cast<const T *>(p.residual) + row * p.residual_stride;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int e = (tid + j * TS) * VEC;
            const bool in = e < p.dim;
            x[j].zero(); z[j].zero(); r[j].zero();
            if (in) x[j].ld(px + e);
            if (in && p.gate) z[j].ld(pz + e);
            if (in && p.residual) r[j].ld(pr + e);
        }
    }
};

// The weights of a thread's channels: kept in registers over the rows (KEEP),
// or read from L2 for every row where the registers are short.
template <int VEC, int CPT, int TS, bool KEEP>
struct Weights {
    const NormParams &p;
    const int tid;
    float kw[KEEP ? CPT : 1][KEEP ? VEC : 1], ks[KEEP ? CPT : 1][KEEP ? VEC : 1], kw2[KEEP ? CPT : 1][KEEP ? VEC : 1];
    __device__ __forceinline__ Weights(const NormParams &p, int tid) : p(p), tid(tid) {
        if constexpr (KEEP)
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    kw[j][c] = post(j, c);
                    ks[j][c] = scaled(j, c);
                    kw2[j][c] = pre(j, c);
                }
    }
    __device__ __forceinline__ int at(int j, int c) const { return (tid + j * TS) * VEC + c; }
    __device__ __forceinline__ float post(int j, int c) const {
        const int e = at(j, c);
        return e < p.dim && p.post_weight ? p.post_weight[p.post_per_channel ? e : e % p.group] : 1.f;
    }
    __device__ __forceinline__ float scaled(int j, int c) const { return at(j, c) < p.dim && p.scale ? p.scale[at(j, c)] : 1.f; }
    __device__ __forceinline__ float pre(int j, int c) const { return at(j, c) < p.dim && p.pre_weight ? p.pre_weight[at(j, c)] : 1.f; }
    __device__ __forceinline__ float w(int j, int c) const { if constexpr (KEEP) return kw[j][c]; else return post(j, c); }
    __device__ __forceinline__ float s(int j, int c) const { if constexpr (KEEP) return ks[j][c]; else return scaled(j, c); }
    __device__ __forceinline__ float w2(int j, int c) const { if constexpr (KEEP) return kw2[j][c]; else return pre(j, c); }
};
// channels a thread can hold all of it for: 1024 threads have 128 registers each
template <int VEC, int CPT, int TS> constexpr bool keep_weights(bool grad) { return CPT * VEC <= (TS == 1024 ? (grad ? 4 : 8) : 16); }

template <typename T, int VEC, int CPT, int TS, bool LDS>
__global__ void __launch_bounds__(TS > 256 ? TS : 256) block_norm_kernel(NormParams p, int mode) {
    constexpr int WG = TS > 256 ? TS : 256, TEAMS = WG / TS, S = LDS ? VEC : 1;
    extern __shared__ float lds[];
    const int tid = threadIdx.x % TS, team = threadIdx.x / TS;
    float *slot = lds + team * team_lds_floats(TS, LDS, p.dim, p.group);
    float *buf = slot + 3 * (TS / 64);
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * TEAMS;
    const Weights<VEC, CPT, TS, keep_weights<VEC, CPT, TS>(false)> w(p, tid);
    RowBuf<T, VEC, CPT, TS> in;
    // every team of a workgroup takes part in every step (the barriers are the
    // workgroup's); a row past the end repeats the last one and writes nothing
    in.load(p, min(first + team, p.rows - 1), tid);
    for (int64_t base = first; base < p.rows; base += step) {
        const int64_t row = base + team;
        const bool live = row < p.rows;
        float a[CPT][VEC], r[CPT][VEC], act[CPT][VEC];
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                a[j][c] = in.x[j].get(c);
                r[j][c] = in.r[j].get(c);
                act[j][c] = 1.f;
                if (p.gate) act[j][c] = gate_act(in.z[j].get(c), p.silu);
            }
        if (base + step < p.rows) in.load(p, min(base + step + team, p.rows - 1), tid);
        if (p.gate && p.gate_first)
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) a[j][c] *= act[j][c];
        if (p.post_weight) {
            float sq[CPT][VEC], q[CPT][S];
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) sq[j][c] = a[j][c] * a[j][c];
            group_sums<VEC, CPT, TS, LDS>(sq, q, p, mode, slot, buf, tid);
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
#pragma unroll
                for (int c = 0; c < S; ++c) q[j][c] = rsqrtf(q[j][c] * p.inv_group + p.eps);
#pragma unroll
                for (int c = 0; c < VEC; ++c) a[j][c] *= q[j][c % S] * w.w(j, c);
            }
        }
        if (p.gate && !p.gate_first)
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) a[j][c] *= act[j][c];
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                a[j][c] = r[j][c] + w.s(j, c) * a[j][c];
                sq += a[j][c] * a[j][c];  // channels past dim hold zeros
            }
        if (live) {
            T *po = static_cast<T *>(p.out) + row * p.dim;
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                const int e = (tid + j * TS) * VEC;
                if (e < p.dim) rowvec<T, VEC>::st(po + e, a[j]);
            }
        }
        if (p.pre_weight) {
            const float q2 = rsqrtf(team_sum<TS>(sq, slot + TS / 64, tid) * p.inv_dim + p.eps);
            T *pn = static_cast<T *>(p.normed) + row * p.dim;
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                const int e = (tid + j * TS) * VEC;
#pragma unroll
                for (int c = 0; c < VEC; ++c) a[j][c] *= q2 * w.w2(j, c);
                if (live && e < p.dim) rowvec<T, VEC>::st(pn + e, a[j]);
            }
        }
        if (TS > 64) lds_barrier();  // the slots are free again
    }
}

// Gradients.  Every team adds its rows' contributions to the weights'
// gradients in registers and writes one row of partial sums at its end,
// [dscale dim | dpre dim | dpost dim or group]; norm_partial_kernel adds the
// teams' rows in a fixed order.
template <typename T, int VEC, int CPT, int TS, bool LDS>
__global__ void __launch_bounds__(TS > 256 ? TS : 256) block_norm_grad_kernel(NormGradParams g, int mode) {
    constexpr int WG = TS > 256 ? TS : 256, TEAMS = WG / TS, S = LDS ? VEC : 1;
    extern __shared__ float lds[];
    const NormParams &p = g.f;
    const int tid = threadIdx.x % TS, team = threadIdx.x / TS;
    float *slot = lds + team * team_lds_floats(TS, LDS || p.group < p.dim, p.dim, p.group);
    float *buf = slot + 3 * (TS / 64);
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * TEAMS;
    constexpr bool AHEAD = keep_weights<VEC, CPT, TS>(true);  // request the next row's vectors early
    const Weights<VEC, CPT, TS, AHEAD> w(p, tid);
    float gw[CPT][VEC] = {}, gs[CPT][VEC] = {}, gw2[CPT][VEC] = {};
    RowBuf<T, VEC, CPT, TS> in;
    rowvec<T, VEC> rdo[CPT], rdn[CPT];
    auto load = [&](int64_t row) {
        in.load(p, row, tid);
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int e = (tid + j * TS) * VEC;
            rdo[j].zero(); rdn[j].zero();
            if (e < p.dim && g.d_out) rdo[j].ld(static_cast<const T *>(g.d_out) + row * p.dim + e);
            if (e < p.dim && g.d_normed) rdn[j].ld(static_cast<const T *>(g.d_normed) + row * p.dim + e);
        }
    };
    if (AHEAD && first < p.rows) load(min(first + team, p.rows - 1));
    for (int64_t base = first; base < p.rows; base += step) {
        const int64_t row = base + team;
        const bool live = row < p.rows;
        if (!AHEAD) load(min(row, p.rows - 1));
        float x[CPT][VEC], r[CPT][VEC], act[CPT][VEC], slope[CPT][VEC], dO[CPT][VEC], dn[CPT][VEC];
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                x[j][c] = in.x[j].get(c);
                r[j][c] = in.r[j].get(c);
                act[j][c] = 1.f; slope[j][c] = 0.f;
                if (p.gate) gate_act_grad(in.z[j].get(c), p.silu, act[j][c], slope[j][c]);
                dO[j][c] = rdo[j].get(c);
                dn[j][c] = rdn[j].get(c);
            }
        if (AHEAD && base + step < p.rows) load(min(base + step + team, p.rows - 1));
        // forward again: hat = a q, v
        float hat[CPT][VEC], q[CPT][S], e1[CPT][VEC];
        const bool first_gate = p.gate && p.gate_first, after_gate = p.gate && !p.gate_first;
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                hat[j][c] = first_gate ? x[j][c] * act[j][c] : x[j][c];
                e1[j][c] = hat[j][c] * hat[j][c];
            }
        if (p.post_weight) {
            group_sums<VEC, CPT, TS, LDS>(e1, q, p, mode, slot, buf, tid);
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
#pragma unroll
                for (int c = 0; c < S; ++c) q[j][c] = rsqrtf(q[j][c] * p.inv_group + p.eps);
#pragma unroll
                for (int c = 0; c < VEC; ++c) hat[j][c] *= q[j][c % S];
            }
        }
        if (p.pre_weight) {
            float s1 = 0.f, s2 = 0.f;
            float out[CPT][VEC];
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    const float v = hat[j][c] * w.w(j, c) * (after_gate ? act[j][c] : 1.f);
                    out[j][c] = r[j][c] + w.s(j, c) * v;
                    s1 += out[j][c] * out[j][c];
                    s2 += dn[j][c] * w.w2(j, c) * out[j][c];
                }
            s1 = wave_sum(s1);
            s2 = wave_sum(s2);
            if (TS > 64) {
                if ((tid & 63) == 0) {
                    slot[TS / 64 + (tid >> 6)] = s1;
                    slot[2 * (TS / 64) + (tid >> 6)] = s2;
                }
                lds_barrier();
                s1 = s2 = 0.f;
#pragma unroll
                for (int k = 0; k < TS / 64; ++k) {
                    s1 += slot[TS / 64 + k];
                    s2 += slot[2 * (TS / 64) + k];
                }
            }
            const float q2 = rsqrtf(s1 * p.inv_dim + p.eps);
            const float k2 = s2 * p.inv_dim * q2 * q2 * q2;
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    dO[j][c] += q2 * dn[j][c] * w.w2(j, c) - out[j][c] * k2;
                    if (live) gw2[j][c] += dn[j][c] * out[j][c] * q2;
                }
        }
        if (live && g.dresidual)
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                const int e = (tid + j * TS) * VEC;
                if (e < p.dim) rowvec<T, VEC>::st(static_cast<T *>(g.dresidual) + row * p.dim + e, dO[j]);
            }
        // through the scale, the gate behind the norm and the norm
        float dz[CPT][VEC];
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float n1 = hat[j][c] * w.w(j, c);
                if (live) gs[j][c] += dO[j][c] * n1 * (after_gate ? act[j][c] : 1.f);
                float dv = dO[j][c] * w.s(j, c);
                dz[j][c] = dv * n1 * slope[j][c];
                if (after_gate) dv *= act[j][c];
                if (live) gw[j][c] += dv * hat[j][c];
                dO[j][c] = dv * w.w(j, c);
                e1[j][c] = dO[j][c] * hat[j][c];
            }
        if (p.post_weight) {
            if (TS > 64 && mode == GROUP_ROW) lds_barrier();  // the first sum's slot is read by now
            float es[CPT][S];
            group_sums<VEC, CPT, TS, LDS>(e1, es, p, mode, slot, buf, tid);
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) dO[j][c] = q[j][c % S] * (dO[j][c] - hat[j][c] * (es[j][c % S] * p.inv_group));
        }
        if (first_gate)
#pragma unroll
            for (int j = 0; j < CPT; ++j)
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    dz[j][c] = dO[j][c] * x[j][c] * slope[j][c];
                    dO[j][c] *= act[j][c];
                }
        if (live)
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
                const int e = (tid + j * TS) * VEC;
                if (e >= p.dim) continue;
                rowvec<T, VEC>::st(static_cast<T *>(g.dx) + row * p.dim + e, dO[j]);
                if (g.dgate) rowvec<T, VEC>::st(static_cast<T *>(g.dgate) + row * p.dim + e, dz[j]);
            }
        if (TS > 64) lds_barrier();  // the slots are free again
    }
    // this team's partial sums; a post_weight shared by the groups has them
    // folded here, in order, through LDS
    const bool fold = g.dpost && !p.post_per_channel && p.group < p.dim;
    float *part = g.partial + (static_cast<int64_t>(blockIdx.x) * TEAMS + team) * norm_partial_cols(p);
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const int e = (tid + j * TS) * VEC + c;
            if (e >= p.dim) continue;
            if (g.dscale) part[e] = gs[j][c];
            if (g.dpre) part[p.dim + e] = gw2[j][c];
            if (fold) buf[e] = gw[j][c];
            else if (g.dpost) part[2 * p.dim + e] = gw[j][c];
        }
    if (fold) {
        lds_barrier();
        for (int e = tid; e < p.group; e += TS) {
            float v = 0.f;
            for (int k = e; k < p.dim; k += p.group) v += buf[k];
            part[2 * p.dim + e] = v;
        }
    }
}

// Column sums of the partial rows: 64 columns a workgroup, NP_ROWS rows at a
// time, a column's partial sums added in order through LDS.
constexpr int NP_ROWS = 16;
__global__ void __launch_bounds__(64 * NP_ROWS) norm_partial_kernel(NormGradParams g, int teams) {
    const NormParams &p = g.f;
    __shared__ float sums[NP_ROWS][64];
    const int lane = threadIdx.x & 63, sub = threadIdx.x >> 6;
    const int blocks_d = (p.dim + 63) / 64;
    const int which = blockIdx.x / blocks_d;  // 0 scale, 1 pre, 2 post
    const int col = (blockIdx.x % blocks_d) * 64 + lane;
    float *to = which == 0 ? g.dscale : which == 1 ? g.dpre : g.dpost;
    if (!to) return;  // the whole workgroup
    const int cols = which == 2 && !p.post_per_channel ? p.group : p.dim;
    const int64_t stride = norm_partial_cols(p);
    float s = 0.f;
    if (col < cols) {
        const float *part = g.partial + which * p.dim + col;
        int t = sub;
        for (; t + 3 * NP_ROWS < teams; t += 4 * NP_ROWS) {  // four rows requested together
            float v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = part[(t + u * NP_ROWS) * stride];
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; t < teams; t += NP_ROWS) s += part[t * stride];
    }
    sums[sub][lane] = s;
    __syncthreads();
    if (sub == 0 && col < cols) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < NP_ROWS; ++k) s += sums[k][lane];
        to[col] = s;
    }
}

bool aligned_rows(const void *ptr, int64_t stride) {
    return !ptr || (reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && stride % 8 == 0);
}

// 128-bit vectors when every row of every plane is aligned for them
bool vector_rows(const NormParams &p) {
    return p.dim % 8 == 0 && aligned_rows(p.x, p.x_stride) && aligned_rows(p.gate, p.gate_stride) &&
           aligned_rows(p.residual, p.residual_stride) && aligned_rows(p.out, 8) && aligned_rows(p.normed, 8);
}

int group_mode(const NormParams &p, int vec) {
    if (p.group == p.dim) return GROUP_ROW;
    const int lanes = p.group / vec;
    if (p.group % vec == 0 && lanes <= 64 && (lanes & (lanes - 1)) == 0) return GROUP_LANES;
    return GROUP_LDS;
}

// Channels per vector, vectors per thread, threads per row.  Forward: 8
// channels a thread.  Gradients: about 24 live values per channel, so 4
// channels a thread, whatever the threads (8192 rows of 4096 channels: 897 us
// with 256 threads of 16 channels, which spill, against 132 us).
struct Shape { int vec, cpt, ts; };
Shape pick(const NormParams &p, bool vec, bool grad) {
    if (!vec) {
        for (int ts : {64, 256, 1024})
            if (p.dim <= 4 * ts) return {1, 4, ts};
        return {1, 16, 1024};
    }
    const int v = grad ? 4 : 8, chunks = p.dim / v;
    for (int ts : {64, 128, 256, 512, 1024})
        if (chunks <= ts) return {v, 1, ts};
    return {v, chunks <= 2048 ? 2 : 4, 1024};
}

template <int V, int C, int TS> struct ShapeC { static constexpr int VEC = V, CPT = C, S = TS; };
template <bool GRAD, typename F>
hipError_t with_shape(const Shape &s, F &&f) {
#define KDA_NORM_CASE(V, C, S) if (s.vec == V && s.cpt == C && s.ts == S) return f(ShapeC<V, C, S>())
    constexpr int V = GRAD ? 4 : 8;
    KDA_NORM_CASE(V, 1, 64); KDA_NORM_CASE(V, 1, 128); KDA_NORM_CASE(V, 1, 256); KDA_NORM_CASE(V, 1, 512);
    KDA_NORM_CASE(V, 1, 1024); KDA_NORM_CASE(V, 2, 1024);
    if constexpr (GRAD) KDA_NORM_CASE(V, 4, 1024);
    KDA_NORM_CASE(1, 4, 64); KDA_NORM_CASE(1, 4, 256); KDA_NORM_CASE(1, 4, 1024); KDA_NORM_CASE(1, 16, 1024);
#undef KDA_NORM_CASE
    return hipErrorInvalidValue;
}

int wg_of(int ts) { return ts > 256 ? ts : 256; }

template <typename T>
hipError_t run_norm(const NormParams &p, hipStream_t s) {
    const Shape sh = pick(p, vector_rows(p), false);
    const int mode = group_mode(p, sh.vec);
    return with_shape<false>(sh, [&](auto shape) {
        constexpr int VEC = decltype(shape)::VEC, CPT = decltype(shape)::CPT, TS = decltype(shape)::S;
        constexpr int WG = TS > 256 ? TS : 256, TEAMS = WG / TS;
        const int64_t want = (p.rows + TEAMS - 1) / TEAMS;
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, 256 * (2048 / WG)));
        const size_t lds = sizeof(float) * TEAMS * team_lds_floats(TS, mode == GROUP_LDS, p.dim, p.group);
        if (mode == GROUP_LDS)
            hipLaunchKernelGGL((block_norm_kernel<T, VEC, CPT, TS, true>), dim3(grid), dim3(WG), lds, s, p, mode);
        else
            hipLaunchKernelGGL((block_norm_kernel<T, VEC, CPT, TS, false>), dim3(grid), dim3(WG), lds, s, p, mode);
        return hipGetLastError();
    });
}

}  // namespace

// Teams the gradient kernel runs: enough waves to fill the chip, no more
// than the rows (each team writes one row of partial sums).
static int grad_teams(const NormParams &p, int ts) {
    const int teams = wg_of(ts) / ts;
    const int64_t want = (p.rows + teams - 1) / teams;
    return static_cast<int>(std::min<int64_t>(want < 1 ? 1 : want, 256 * (1024 / wg_of(ts)))) * teams;
}

// The workspace must hold the partial rows of either path (which one runs
// depends on addresses, which the size query does not know).
size_t block_norm_grad_bytes(const NormParams &p) {
    int teams = grad_teams(p, pick(p, false, true).ts);
    if (p.dim % 8 == 0) teams = std::max(teams, grad_teams(p, pick(p, true, true).ts));
    return align_up(sizeof(float) * static_cast<size_t>(teams) * norm_partial_cols(p));
}

hipError_t launch_block_norm(const NormParams &p, int dtype, hipStream_t s) {
    return dtype == 0 ? run_norm<float>(p, s) : run_norm<bf16_t>(p, s);
}

template <typename T>
static hipError_t run_norm_grad(const NormGradParams &g, hipStream_t s) {
    const NormParams &p = g.f;
    bool vec = vector_rows(p);
    for (const void *ptr : {g.d_out, g.d_normed, static_cast<const void *>(g.dx), static_cast<const void *>(g.dgate),
                            static_cast<const void *>(g.dresidual)})
        vec = vec && aligned_rows(ptr, 8);
    const Shape sh = pick(p, vec, true);
    const int mode = group_mode(p, sh.vec);
    const int teams = grad_teams(p, sh.ts);
    hipError_t e = with_shape<true>(sh, [&](auto shape) {
        constexpr int VEC = decltype(shape)::VEC, CPT = decltype(shape)::CPT, TS = decltype(shape)::S;
        constexpr int WG = TS > 256 ? TS : 256, TEAMS = WG / TS;
        const size_t lds = sizeof(float) * TEAMS * team_lds_floats(TS, mode == GROUP_LDS || p.group < p.dim, p.dim, p.group);
        if (mode == GROUP_LDS)
            hipLaunchKernelGGL((block_norm_grad_kernel<T, VEC, CPT, TS, true>), dim3(teams / TEAMS), dim3(WG), lds, s, g, mode);
        else
            hipLaunchKernelGGL((block_norm_grad_kernel<T, VEC, CPT, TS, false>), dim3(teams / TEAMS), dim3(WG), lds, s, g, mode);
        return hipGetLastError();
    });
    if (e != hipSuccess || !(g.dscale || g.dpre || g.dpost)) return e;
    hipLaunchKernelGGL(norm_partial_kernel, dim3(3 * ((p.dim + 63) / 64)), dim3(64 * NP_ROWS), 0, s, g, teams);
    return hipGetLastError();
}

hipError_t launch_block_norm_grad(const NormGradParams &g, int dtype, hipStream_t s) {
    return dtype == 0 ? run_norm_grad<float>(g, s) : run_norm_grad<bf16_t>(g, s);
}

}  // namespace kda
