// Gradients of the short causal convolution (include/kda.h).  With
//     pre_t = bias + sum_j w_j x_{t-W+1+j},   g_t = dy_t act'(pre_t):
//     dx_t  = sum_j w_j g_{t+W-1-j}  (+ d_final of the last W - 1 tokens),
//     dw_j  = sum_t g_t x_{t-W+1+j},  dbias = sum_t g_t,
//     d_initial: the same sum as dx at the W - 1 places before the sequence.
// act'(pre) = s + pre s (1 - s) with s = sigmoid(pre); pre is recomputed.
//
// HBM-bound: x and dy are read once and dx written once.  A thread owns 4
// neighbouring channels and walks a tile of consecutive tokens with the last
// W - 1 inputs and the W unfinished sums of dx in registers: g_t adds w_j g_t
// to the sum of the token W - 1 - j places back, and the oldest sum is
// complete.  It walks W - 1 tokens past its tile to finish the tile's sums (x
// and dy of those come from L2: the neighbouring thread reads them too).  Four
// tokens are requested while the four before are worked on, and tokens whose
// windows lie inside one sequence take a path without branches.  The sums over
// tokens of dw and dbias stay in registers, the threads of a workgroup that
// share channels add theirs through LDS, and every workgroup writes one row of
// partial sums; a second kernel adds the rows in order.
//
// 2 x 4096 tokens of 4096 bf16 channels, W = 4, SiLU: 53 us for this kernel
// (3.8 TB/s; a copy of the same bytes takes 39), 61 in all.  8 channels a
// thread with 16-byte requests took 68 (229 registers, 2 waves a SIMD; 4
// channels need 144), tiles of 32 tokens 60; held to 128 registers it spills
// (120).  About 36 vector instructions a value (counted) issue in 31 to
// 36 us of it; the rest is waiting, at 3 waves a SIMD.
#include "kda_launch.hpp"

namespace kda {

namespace {

constexpr int CG_THREADS = 256, CPT = 4;

template <typename T> struct chvec;  // CPT channels
template <> struct chvec<bf16_t> {
    uint2 u;
    __device__ __forceinline__ void ld(const bf16_t *p) { u = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
    __device__ __forceinline__ float get(int c) const {
        const uint32_t w = c < 2 ? u.x : u.y;
        return __uint_as_float((c & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ __forceinline__ static void st(bf16_t *p, const float (&v)[CPT]) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = static_cast<uint32_t>(f32_to_bf16(v[2 * i])) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
};
template <> struct chvec<float> {
    f32x4 u;
    __device__ __forceinline__ void ld(const float *p) { u = *reinterpret_cast<const f32x4 *>(p); }
    __device__ __forceinline__ void zero() { u = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ float get(int c) const { return u[c]; }
    __device__ __forceinline__ static void st(float *p, const float (&v)[CPT]) {
        *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
    }
};

// act'(pre) dy
__device__ __forceinline__ float through_act(float pre, float dy, int silu) {
    if (!silu) return dy;
    const float s = __builtin_amdgcn_rcpf(1.f + fast_exp2(-pre * kLog2e));  // exp2 overflows to inf: s = 0
    // pre s is 0 where s is, also for pre = -inf
    const float ps = s > 0.f ? pre * s : 0.f;
    return dy * fmaf(ps, 1.f - s, s);
}

// Sequence holding token t: as the forward's conv_seq, any contents of
// cu_seqlens give start <= t < end inside [0, ntok].
struct ConvSeq { int n, start, end; };
__device__ __forceinline__ ConvSeq grad_seq(const ConvGradParams &p, int t) {
    ConvSeq s;
    if (!p.cu_seqlens) {
        s.n = t / p.T;
        s.start = s.n * p.T;
        s.end = s.start + p.T;
        return s;
    }
    int lo = 0, hi = p.N;  // last n with cu[n] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
    }
    s.n = lo;
    s.start = min(max(p.cu_seqlens[lo], 0), t);
    s.end = max(min(p.cu_seqlens[lo + 1], p.B * p.T), t + 1);
    return s;
}

// input `back` >= 1 places before the start of sequence n
__device__ __forceinline__ float before_start(const ConvGradParams &p, int n, int c, int back) {
    return p.initial_state ? p.initial_state[(static_cast<int64_t>(n) * p.C + c) * (p.W - 1) + (p.W - 1 - back)] : 0.f;
}

// LG threads side by side on channel vectors, CG_THREADS / LG tiles of tt
// tokens one below the other.
template <typename TI, typename TG, int W>
__global__ void __launch_bounds__(CG_THREADS) conv_grad_kernel(ConvGradParams p, int LG, int tt, int cols) {
    constexpr int HW = W - 1;
    extern __shared__ float red[];  // [waves][CPT (W + 1)][LG] at the end
    const int lane = threadIdx.x % LG, sub = threadIdx.x / LG, subs = CG_THREADS / LG;
    const int c0 = ((blockIdx.x % cols) * LG + lane) * CPT;
    const bool on = c0 < p.C;
    const int ntok = p.B * p.T;
    const int64_t t_first = (static_cast<int64_t>(blockIdx.x / cols) * subs + sub) * tt;
    const TI *x = static_cast<const TI *>(p.x);
    const TG *dy = static_cast<const TG *>(p.d_y);
    TI *dx = static_cast<TI *>(p.dx);
    float dw[CPT][W] = {}, db[CPT] = {};
    if (on && t_first < ntok) {
        const int t0 = static_cast<int>(t_first), t1 = min(t0 + tt, ntok);
        float w[CPT][W], bias[CPT];
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[c][j] = p.weight[static_cast<int64_t>(c0 + c) * W + j];
            bias[c] = p.bias ? p.bias[c0 + c] : 0.f;
        }
        ConvSeq sq = grad_seq(p, t0);
        // window: xs[c][j] = input of place t - HW + j; acc[c][j]: unfinished dx of the same place
        float xs[CPT][W], acc[CPT][W];
#pragma unroll
        for (int j = 0; j < HW; ++j) {
            const int pos = t0 - HW + j;
            chvec<TI> v;
            v.zero();
            if (pos >= sq.start) v.ld(x + static_cast<int64_t>(pos) * p.C + c0);
#pragma unroll
            for (int c = 0; c < CPT; ++c) xs[c][j] = pos >= sq.start ? v.get(c) : before_start(p, sq.n, c0 + c, sq.start - pos);
        }
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
            for (int j = 0; j < W; ++j) acc[c][j] = 0.f;
        const int t_end = t1 + HW;  // the last W - 1 steps only finish sums
        constexpr int U = 4;        // tokens whose x and dy are requested together, ahead of their use
        chvec<TI> xv[U], xn[U];
        chvec<TG> gv[U], gn[U];
        auto request = [&](int tb, chvec<TI> (&xq)[U], chvec<TG> (&gq)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = static_cast<int64_t>(min(tb + u, ntok - 1)) * p.C + c0;  // past the end g is set to 0
                xq[u].ld(x + at);
                gq[u].ld(dy + at);
            }
        };
        request(t0, xv, gv);
        for (int tb = t0; tb < t_end; tb += U) {
            request(tb + U, xn, gn);
            if (tb + U <= min(t1, sq.end) && tb - sq.start >= HW) {
                // own tokens of one sequence, whose windows lie inside it; its
                // end, where d_final is added, is W - 1 tokens off
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int c = 0; c < CPT; ++c) {
                        xs[c][HW] = xv[u].get(c);
                        float pre = bias[c];
#pragma unroll
                        for (int j = 0; j < W; ++j) pre = fmaf(w[c][j], xs[c][j], pre);
                        const float g = through_act(pre, gv[u].get(c), p.silu);
                        db[c] += g;
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            dw[c][j] = fmaf(g, xs[c][j], dw[c][j]);
                            acc[c][j] = fmaf(w[c][j], g, acc[c][j]);
                        }
                    }
                    if (tb + u - HW >= t0) {
                        float out[CPT];
#pragma unroll
                        for (int c = 0; c < CPT; ++c) out[c] = acc[c][0];
                        chvec<TI>::st(dx + static_cast<int64_t>(tb + u - HW) * p.C + c0, out);
                    }
#pragma unroll
                    for (int c = 0; c < CPT; ++c) {
#pragma unroll
                        for (int j = 0; j < HW; ++j) {
                            xs[c][j] = xs[c][j + 1];
                            acc[c][j] = acc[c][j + 1];
                        }
                        acc[c][HW] = 0.f;
                    }
                }
            } else
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = tb + u;
                if (t >= t_end) break;
                if (t >= sq.end && t < ntok) {  // a sequence starts at t
                    sq = grad_seq(p, t);
#pragma unroll
                    for (int j = 0; j < HW; ++j)
#pragma unroll
                        for (int c = 0; c < CPT; ++c) xs[c][j] = before_start(p, sq.n, c0 + c, HW - j);
                }
                const bool own = t < t1;
                const int reach = t - sq.start;  // places of this sequence before t
                float g[CPT];
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    xs[c][HW] = xv[u].get(c);
                    float pre = bias[c];
#pragma unroll
                    for (int j = 0; j < W; ++j) pre = fmaf(w[c][j], xs[c][j], pre);
                    g[c] = through_act(pre, gv[u].get(c), p.silu);
                    if (t >= ntok) g[c] = 0.f;
                    if (own) {
                        db[c] += g[c];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[c][j] = fmaf(g[c], xs[c][j], dw[c][j]);
                    }
                }
                if (reach >= HW) {
#pragma unroll
                    for (int c = 0; c < CPT; ++c)
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[c][j] = fmaf(w[c][j], g[c], acc[c][j]);
                } else {  // places before the sequence belong to another one
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (HW - j <= reach)
#pragma unroll
                            for (int c = 0; c < CPT; ++c) acc[c][j] = fmaf(w[c][j], g[c], acc[c][j]);
                }
                const int done = t - HW;  // its sum is complete
                if (done >= t0 && done < t1) {
                    float out[CPT];
#pragma unroll
                    for (int c = 0; c < CPT; ++c) out[c] = acc[c][0];
                    if (p.d_final && HW > 0) {
                        const ConvSeq ds = done >= sq.start && done < sq.end ? sq : grad_seq(p, done);
                        const int k = done - (ds.end - HW);
                        if (k >= 0)
#pragma unroll
                            for (int c = 0; c < CPT; ++c) out[c] += p.d_final[(static_cast<int64_t>(ds.n) * p.C + c0 + c) * HW + k];
                    }
                    chvec<TI>::st(dx + static_cast<int64_t>(done) * p.C + c0, out);
                }
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
#pragma unroll
                    for (int j = 0; j < HW; ++j) {
                        xs[c][j] = xs[c][j + 1];
                        acc[c][j] = acc[c][j + 1];
                    }
                    acc[c][HW] = 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) { xv[u] = xn[u]; gv[u] = gn[u]; }
        }
    }
    // one row of partial sums per workgroup, [dw C W | dbias C]: lanes of a
    // wave that share channels add theirs by exchanges, the waves through LDS
    constexpr int NV = CPT * (W + 1);
    const int wave = threadIdx.x >> 6, wl = threadIdx.x & 63;
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int j = 0; j <= W; ++j) {
            float v = j < W ? dw[c][j < W ? j : 0] : db[c];
            for (int m = LG; m < 64; m <<= 1) v += __shfl_xor(v, m);
            if (wl < LG) red[(wave * NV + c * (W + 1) + j) * LG + wl] = v;
        }
    lds_barrier();
    float *part = p.partial + static_cast<int64_t>(blockIdx.x / cols) * p.C * (W + 1);
    for (int i = threadIdx.x; i < NV * LG; i += CG_THREADS) {
        const int v = i / LG, cv = (blockIdx.x % cols) * LG + i % LG;
        const int ch = cv * CPT + v / (W + 1), j = v % (W + 1);
        if (ch >= p.C) continue;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < CG_THREADS / 64; ++k) sum += red[k * NV * LG + i];
        part[j < W ? static_cast<int64_t>(ch) * W + j : static_cast<int64_t>(p.C) * W + ch] = sum;
    }
}

// Adds the rows of partial sums: 64 columns a workgroup, 4 row strides.
__global__ void __launch_bounds__(256) conv_grad_sum_kernel(ConvGradParams p, int rows) {
    __shared__ float s[4][64];
    const int64_t cols = static_cast<int64_t>(p.C) * (p.W + 1);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
    const int sub = threadIdx.x >> 6;
    float v = 0.f;
    if (col < cols)
        for (int r = sub; r < rows; r += 4) v += p.partial[r * cols + col];
    s[sub][threadIdx.x & 63] = v;
    __syncthreads();
    if (sub == 0 && col < cols) {
        v = (s[0][threadIdx.x] + s[1][threadIdx.x]) + (s[2][threadIdx.x] + s[3][threadIdx.x]);
        if (col < static_cast<int64_t>(p.C) * p.W) p.dweight[col] = v;
        else if (p.dbias) p.dbias[col - static_cast<int64_t>(p.C) * p.W] = v;
    }
}

// d_initial[n][c][k], the place W - 1 - k before the sequence: from the g of
// the first W - 1 tokens, and d_final where the sequence is shorter than that.
template <typename TI, typename TG, int W>
__global__ void __launch_bounds__(CG_THREADS) conv_grad_state_kernel(ConvGradParams p) {
    constexpr int HW = W - 1;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * CG_THREADS + threadIdx.x;
    if (item >= static_cast<int64_t>(p.N) * p.C) return;
    const int n = static_cast<int>(item / p.C), c = static_cast<int>(item % p.C);
    const int ntok = p.B * p.T;
    int start = n * p.T, end = start + p.T;
    if (p.cu_seqlens) {
        start = min(max(p.cu_seqlens[n], 0), ntok);
        end = min(max(p.cu_seqlens[n + 1], start), ntok);
    }
    const int len = end - start;
    float in[2 * HW + 1], w[W], d[HW + 1];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = p.weight[static_cast<int64_t>(c) * W + j];
#pragma unroll
    for (int k = 0; k < HW; ++k) {
        in[k] = before_start(p, n, c, HW - k);
        in[HW + k] = k < len ? io<TI>::ld(static_cast<const TI *>(p.x), static_cast<int64_t>(start + k) * p.C + c) : 0.f;
        // the final state of a sequence of len tokens holds this place at k - len
        d[k] = k >= len && p.d_final ? p.d_final[item * HW + k - len] : 0.f;
    }
    const float bias = p.bias ? p.bias[c] : 0.f;
#pragma unroll
    for (int t = 0; t < HW; ++t) {
        if (t >= len) continue;
        float pre = bias;
#pragma unroll
        for (int j = 0; j < W; ++j) pre = fmaf(w[j], in[t + j], pre);
        const float g = through_act(pre, io<TG>::ld(static_cast<const TG *>(p.d_y), static_cast<int64_t>(start + t) * p.C + c), p.silu);
#pragma unroll
        for (int k = t; k < HW; ++k) d[k] = fmaf(w[k - t], g, d[k]);  // place t + j of the window, j = k - t
    }
#pragma unroll
    for (int k = 0; k < HW; ++k) p.d_initial[item * HW + k] = d[k];
}

struct ConvGrid { int lg, tt, rows, cols; };
// Channel vectors side by side: the most of {64, 32, 16, 8} that wastes at
// most an eighth of the lanes (8 lanes still make 64- or 128-byte pieces),
// fewer only where there are fewer.
// Tokens per thread: 64, fewer while that leaves CUs without a workgroup (the
// walk past the tile then costs more of it).
ConvGrid conv_grid(const ConvGradParams &p) {
    ConvGrid g;
    const int vecs = p.C / CPT;
    for (g.lg = 1; g.lg < 8 && g.lg < vecs;) g.lg *= 2;
    for (int lg : {64, 32, 16}) {
        const int padded = (vecs + lg - 1) / lg * lg;
        if ((padded - vecs) * 8 <= padded) { g.lg = lg; break; }
    }
    g.cols = (vecs + g.lg - 1) / g.lg;
    const int subs = CG_THREADS / g.lg;
    const int64_t ntok = static_cast<int64_t>(p.B) * p.T;
    g.tt = 64;
    while (g.tt > 8 && (ntok + static_cast<int64_t>(subs) * g.tt - 1) / (static_cast<int64_t>(subs) * g.tt) * g.cols < 512) g.tt /= 2;
    g.rows = static_cast<int>((ntok + static_cast<int64_t>(subs) * g.tt - 1) / (static_cast<int64_t>(subs) * g.tt));
    return g;
}

template <typename TI, typename TG, int W>
hipError_t run(const ConvGradParams &p, hipStream_t s) {
    const ConvGrid g = conv_grid(p);
    if (g.rows > 0) {
        hipLaunchKernelGGL((conv_grad_kernel<TI, TG, W>), dim3(static_cast<unsigned>(g.cols) * g.rows), dim3(CG_THREADS),
                           sizeof(float) * (CG_THREADS / 64) * CPT * (W + 1) * g.lg, s, p, g.lg, g.tt, g.cols);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t cols = static_cast<int64_t>(p.C) * (W + 1);
    hipLaunchKernelGGL(conv_grad_sum_kernel, dim3(static_cast<unsigned>((cols + 63) / 64)), dim3(256), 0, s, p, g.rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.d_initial || W == 1 || p.N == 0) return e;
    const int64_t items = static_cast<int64_t>(p.N) * p.C;
    hipLaunchKernelGGL((conv_grad_state_kernel<TI, TG, W>), dim3(static_cast<unsigned>((items + CG_THREADS - 1) / CG_THREADS)),
                       dim3(CG_THREADS), 0, s, p);
    return hipGetLastError();
}

template <typename TI, typename TG>
hipError_t run_w(const ConvGradParams &p, hipStream_t s) {
    switch (p.W) {
        case 1: return run<TI, TG, 1>(p, s);
        case 2: return run<TI, TG, 2>(p, s);
        case 3: return run<TI, TG, 3>(p, s);
        case 4: return run<TI, TG, 4>(p, s);
        case 5: return run<TI, TG, 5>(p, s);
        case 6: return run<TI, TG, 6>(p, s);
        case 7: return run<TI, TG, 7>(p, s);
        default: return run<TI, TG, 8>(p, s);
    }
}
}  // namespace

size_t conv_grad_bytes(const ConvGradParams &p) {
    const int64_t rows = conv_grid(p).rows;
    return align_up(sizeof(float) * static_cast<size_t>(rows < 1 ? 1 : rows) * p.C * (p.W + 1));
}

hipError_t launch_short_conv_grad(const ConvGradParams &p, int in_dtype, int grad_dtype, hipStream_t s) {
    if (in_dtype == 0 && grad_dtype == 0) return run_w<float, float>(p, s);
    if (in_dtype == 0 && grad_dtype == 1) return run_w<float, bf16_t>(p, s);
    if (in_dtype == 1 && grad_dtype == 0) return run_w<bf16_t, float>(p, s);
    return run_w<bf16_t, bf16_t>(p, s);
}

}  // namespace kda
