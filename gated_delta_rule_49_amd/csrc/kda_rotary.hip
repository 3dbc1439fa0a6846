// Rotary positions on part of each head, and the write of new tokens into the
// paged latent cache (norm of the latent, rotation of the shared key).
#include "kda_latent.hpp"

namespace kda {

namespace {

// V values of 16 bytes, or one
template <typename T, int V> struct vec {
    float x[V];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (V == 1) {
            x[0] = io<T>::ld(p, 0);
        } else if constexpr (sizeof(T) == 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = v[i];
        } else {
            frag8 f;
            f.u = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = bf16_to_f32(f.s[i]);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (V == 1) {
            io<T>::st(p, 0, x[0]);
        } else if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4 *>(p) = f32x4{x[0], x[1], x[2], x[3]};
        } else {
            frag8 f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f.s[i] = f32_to_bf16(x[i]);
            *reinterpret_cast<uint4 *>(p) = f.u;
        }
    }
};

// One workgroup takes one token, or as many as fill its threads: the angles of
// their pairs once, in LDS, for all heads; then the heads' channels in units of
// one vector (copied channels, interleaved pairs) or of two, half the rotated part
// apart.  Bound by memory: 32768 tokens of 32 heads of 192 channels, 64 of them
// turned, bf16, in 144 us (5.6 TB/s).
constexpr int kRotThreads = 256, kRotPairs = 512;
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(RotaryParams p, int copies, uint32_t units, int group) {
    __shared__ float s_cos[kRotPairs], s_sin[kRotPairs];
    const int64_t first = p.start + static_cast<int64_t>(blockIdx.x) * group;
    const int count = static_cast<int>(min(static_cast<int64_t>(group), static_cast<int64_t>(p.B) * p.T - first));
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < count * pairs; i += kRotThreads) {
        const int64_t bt = first + i / pairs;
        const int b = static_cast<int>(bt / p.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * p.T);
        const double pos = p.pos ? p.pos[b * p.p_sb + t * p.p_st] : t;
        float sn, cs;
        sincos_far(pos * p.freqs[i % pairs], sn, cs);
        s_cos[i] = cs * p.magnitude;
        s_sin[i] = (p.back ? -sn : sn) * p.magnitude;
    }
    __syncthreads();
    const uint32_t each = units * p.H, total = each * count;
    for (uint32_t e = threadIdx.x; e < total; e += kRotThreads) {
        const uint32_t g = group == 1 ? 0 : e / each, i = e - g * each;
        const int64_t bt = first + g;
        const int b = static_cast<int>(bt / p.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * p.T);
        const T *x = static_cast<const T *>(p.x) + b * p.x_sb + t * p.x_st;
        T *out = static_cast<T *>(p.out) + b * p.o_sb + t * p.o_st;
        const float *cosines = s_cos + g * pairs, *sines = s_sin + g * pairs;
        const uint32_t h = i / units, u = i - h * units;
        const T *xh = x + h * p.x_sh;
        T *oh = out + h * p.o_sh;
        if (static_cast<int>(u) < copies) {  // channels that do not turn
            const int c = static_cast<int>(u) * V, at = c < p.offset ? c : c + p.rot;
            vec<T, V> a;
            a.load(xh + at);
            a.store(oh + at);
            continue;
        }
        const int k = static_cast<int>(u) - copies;
        vec<T, V> a, d;
        if constexpr (INTER && V > 1) {
            const int at = p.offset + k * V;
            a.load(xh + at);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const float cs = cosines[k * (V / 2) + j], sn = sines[k * (V / 2) + j];
                d.x[2 * j] = a.x[2 * j] * cs - a.x[2 * j + 1] * sn;
                d.x[2 * j + 1] = a.x[2 * j] * sn + a.x[2 * j + 1] * cs;
            }
            d.store(oh + at);
        } else {
            const int at = p.offset + (INTER ? 2 * k : k * V), other = at + (INTER ? 1 : pairs);
            a.load(xh + at);
            d.load(xh + other);
            vec<T, V> e;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float cs = cosines[k * V + j], sn = sines[k * V + j];
                e.x[j] = a.x[j] * cs - d.x[j] * sn;
                d.x[j] = a.x[j] * sn + d.x[j] * cs;
            }
            e.store(oh + at);
            d.store(oh + other);
        }
    }
}

template <typename T, int V, bool INTER>
hipError_t run_rotary(const RotaryParams &p, hipStream_t s) {
    const bool in_place = p.x == p.out;
    const int copies = in_place ? 0 : (p.D - p.rot) / V;
    const int turned = V == 1 || !INTER ? p.rot / 2 / V : p.rot / V;
    if (copies + turned == 0) return hipSuccess;
    const int64_t tokens = static_cast<int64_t>(p.B) * p.T, each = static_cast<int64_t>(copies + turned) * p.H;
    const int64_t group = std::max<int64_t>(1, std::min<int64_t>(kRotThreads / each, p.rot ? 2 * kRotPairs / p.rot : kRotThreads));
    // a launch has fewer than 2^32 threads
    const int64_t most = 1 << 23, slice = most * group;
    for (RotaryParams q = p; q.start < tokens; q.start += slice) {
        const unsigned grid = static_cast<unsigned>(std::min(most, (tokens - q.start + group - 1) / group));
        rotary_kernel<T, V, INTER><<<grid, kRotThreads, 0, s>>>(q, copies, copies + turned, static_cast<int>(group));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <typename T>
hipError_t pick_rotary(const RotaryParams &p, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    bool wide = (reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) % 16 == 0 && p.offset % V == 0 && p.D % V == 0 &&
                (p.interleaved ? p.rot : p.rot / 2) % V == 0;
    for (const int64_t st : {p.x_sb, p.x_st, p.x_sh, p.o_sb, p.o_st, p.o_sh}) wide = wide && st % V == 0;
    if (wide) return p.interleaved ? run_rotary<T, V, true>(p, s) : run_rotary<T, V, false>(p, s);
    return p.interleaved ? run_rotary<T, 1, true>(p, s) : run_rotary<T, 1, false>(p, s);
}

// One wave a token.  The row is held in registers between the sum of squares
// and the write (NV vectors a lane).  The sequence of a packed token is found
// by 64 probes at a time: two rounds up to 4096 sequences.  256 tokens of 512 + 64
// channels take 4.3 us (latency: offsets, length, page, row), 17588 packed ones
// 14.7 us (4.1 TB/s of rows read and written).
template <typename T, int NV>
__global__ void __launch_bounds__(256) append_kernel(LatentAppendParams p) {
    constexpr int V = 16 / sizeof(T);
    const int64_t token = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (token >= static_cast<int64_t>(p.B) * p.T) return;
    int n, t;  // sequence, place in it
    bool mine = true;
    const T *row;
    if (p.cu) {
        row = static_cast<const T *>(p.kv) + token * p.kv_st;
        int lo = 0, hi = p.N;  // the last n in [lo, hi) with cu[n] <= token
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) / 64;
            const int at = lo + lane * step;
            const bool below = at < hi && p.cu[at] <= token;
            const int found = 63 - __clzll(static_cast<long long>(__ballot(below) | 1ull));
            lo += found * step;
            hi = min(hi, lo + step);
        }
        n = lo;
        const int32_t begin = p.cu[n], end = p.cu[n + 1];
        mine = token >= begin && token < end;  // else before the first sequence or behind the last
        t = static_cast<int>(token - begin);
    } else {
        n = static_cast<int>(token / p.T);
        t = static_cast<int>(token - static_cast<int64_t>(n) * p.T);
        row = static_cast<const T *>(p.kv) + n * p.kv_sb + t * p.kv_st;
    }
    const int64_t pos = static_cast<int64_t>(p.lengths[n]) + t;
    vec<T, V> a[NV];
    float square = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 64 + lane) * V;
        if (c >= p.dc) continue;
        a[i].load(row + c);
#pragma unroll
        for (int j = 0; j < V; ++j) square = fmaf(a[i].x[j], a[i].x[j], square);
    }
    T *to = nullptr;
    const int64_t page = mine && pos >= 0 ? pos / p.page_size : -1;
    if (page >= 0 && page < p.max_pages) {
        const int32_t id = p.page_table[n * p.table_stride + page];
        if (id >= 0 && id < p.num_pages)
            to = static_cast<T *>(p.cache) + id * p.page_stride + (pos - page * p.page_size) * p.row_stride;
    }
    if (!to && mine && p.status && lane == 0) *p.status = kBadPages;  // any writer writes the same
    T *copy = p.rows && mine ? static_cast<T *>(p.rows) + token * (p.dc + p.dr) : nullptr;
    float inv = 1.f;
    if (p.weight) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) square += __shfl_xor(square, d);
        inv = 1.f / sqrtf(square / static_cast<float>(p.dc) + p.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 64 + lane) * V;
        if (c >= p.dc) continue;
        if (p.weight) {
#pragma unroll
            for (int j = 0; j < V; ++j) a[i].x[j] = a[i].x[j] * inv * p.weight[c + j];
        }
        if (to) a[i].store(to + c);
        if (copy) a[i].store(copy + c);
    }
    // one lane a pair: neighbours, or half of d_rope apart
    const int pairs = p.dr / 2;
    for (int i = lane; i < pairs; i += 64) {
        const int c0 = p.dc + (p.interleaved ? 2 * i : i), c1 = c0 + (p.interleaved ? 1 : pairs);
        float x = io<T>::ld(row, c0), y = io<T>::ld(row, c1);
        if (p.freqs) {
            float sn, cs;
            sincos_far(static_cast<double>(pos) * p.freqs[i], sn, cs);
            const float u = p.magnitude * (x * cs - y * sn);
            y = p.magnitude * (x * sn + y * cs);
            x = u;
        }
        if (to) { io<T>::st(to, c0, x); io<T>::st(to, c1, y); }
        if (copy) { io<T>::st(copy, c0, x); io<T>::st(copy, c1, y); }
    }
}

template <typename T>
hipError_t pick_append(const LatentAppendParams &p, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.B) * p.T + 3) / 4);
    const int need = (p.dc + 64 * V - 1) / (64 * V);
    if (need <= 1) append_kernel<T, 1><<<grid, 256, 0, s>>>(p);
    else if (need <= 2) append_kernel<T, 2><<<grid, 256, 0, s>>>(p);
    else if (need <= 4) append_kernel<T, 4><<<grid, 256, 0, s>>>(p);
    else append_kernel<T, 8><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryParams &p, int dtype, hipStream_t s) {
    return dtype == 0 ? pick_rotary<float>(p, s) : pick_rotary<bf16_t>(p, s);
}
hipError_t launch_latent_append(const LatentAppendParams &p, int dtype, hipStream_t s) {
    return dtype == 0 ? pick_append<float>(p, s) : pick_append<bf16_t>(p, s);
}

}  // namespace kda
