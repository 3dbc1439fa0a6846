// Latent attention on the bf16 matrix cores: what the forward and the gradients
// share.
//
// v_mfma_f32_32x32x16_bf16: A is 32 x 16, lane l holds row l % 32 and the 8
// contraction slots of half l / 32; B likewise by columns; C/D: lane l holds
// column l % 32, register i row 8 (i / 4) + 4 (l / 32) + i % 4.  Sixteen rows of
// a C tile, from row 16 s, are its registers 8 s .. 8 s + 7: converted to bf16
// they are the B operand of the next product as they stand, when that product's
// A operand takes the same rows in its slots: 4 h .. 4 h + 3 and 8 + 4 h .. of
// them for half h.  So P and dS never leave their lanes.
//
// LDS tiles are row-major bf16, rows of D channels cut into chunks of 16 bytes
// that are permuted inside the row.  Two ways to read them:
//   by rows   16 bytes of row l % 32: chunk c of row r lies at c ^ s(r), with
//             s(r) such that 8 rows in a row, and 16, fall on different banks
//   by columns   ds_read_b64_tr_b16, four rows by 16 channels for each 16 lanes:
//             pairs of chunks u of row r lie at u ^ f(r % 4), f = 0, 3, 5, 6 (for
//             128 channels), so that the four rows' 32 bytes fall on different banks
#pragma once
#include "kda_latent.hpp"

namespace kda {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

__device__ __forceinline__ f32x16 mfma32(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// registers 8 s .. 8 s + 7 of a C tile as an operand
__device__ __forceinline__ bf16x8 half_tile(const f32x16 &c, int s) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = static_cast<__bf16>(c[8 * s + i]);
    return r;
}

__device__ __forceinline__ uint2 read_tr16(const char *at) {
    const v4i16 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(at));
    return __builtin_bit_cast(uint2, r);
}

__device__ __forceinline__ float swap_halves_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float swap_halves_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// How a tile's chunks are permuted: the byte of chunk c of row r in a tile of D
// channels.  Each permutation is its own inverse within the row.
struct RowRead {  // read by rows
    template <int D> __device__ __forceinline__ static constexpr int place(int r, int c) {
        if constexpr (D == 128) return r * (D * 2) + ((c ^ (r & 15)) * 16);
        else return r * (D * 2) + ((c & ~7) * 16) + (((c ^ r ^ (r >> 3 & 1)) & 7) * 16);
    }
};
struct ColumnRead {  // read by columns
    template <int D> __device__ __forceinline__ static constexpr int place(int r, int c) {
        const int t = r & 3;
        if constexpr (D == 64) return r * (D * 2) + ((c ^ (t << 1)) * 16);
        else return r * (D * 2) + ((c ^ (((t << 1) ^ ((t ^ (t >> 1)) & 1)) << 1)) * 16);
    }
};
struct BothRead {  // read in both ways
    template <int D> __device__ __forceinline__ static constexpr int place(int r, int c) {
        return r * (D * 2) + ((c & ~7) * 16) + (((c ^ r ^ (r >> 3 & 1)) & 7) * 16);
    }
    // A lane's place for the first 16 channels of row c32, by rows; k 16-channel steps further
    template <int D> __device__ __forceinline__ static uint32_t row(int lane) { return place<D>(lane & 31, lane >> 5); }
    __device__ __forceinline__ static uint32_t step(uint32_t at, int k) { return (at ^ (32 * (k & 3))) + (k >> 2) * 128; }
    // .. and for 32 channels of 16 rows, by columns: rows 4 h + 0..3 and 8 rows on; block b of channels
    template <int D> __device__ __forceinline__ static uint32_t columns(int lane) {
        return place<D>(4 * (lane >> 5) + ((lane & 15) >> 2), 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) + 8 * (lane & 1);
    }
    template <int D> __device__ __forceinline__ static bf16x8 read_columns(const char *tile, uint32_t at, int b) {
        const char *from = tile + (b >> 1) * 128;
        const uint32_t turned = at ^ (64 * (b & 1));
        const uint2 lo = read_tr16(from + turned), hi = read_tr16(from + 8 * D * 2 + (turned ^ 16));
        frag8 f;
        f.u = make_uint4(lo.x, lo.y, hi.x, hi.y);
        return f.v;
    }
};

// 16 bytes a lane from memory to LDS without a register between: lane i's go to
// `to` + 16 i (`to` the wave's own, the same in all its lanes).  Written in
// assembly because the compiler, which cannot tell the tiles apart, would wait
// for the next tile's loads before any read of this one.  There is no output
// register, and the wait is the caller's: wait_loads(), then a barrier.
__device__ __forceinline__ void load_to_lds(const void *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory");
}
// .. and 4 bytes a lane
__device__ __forceinline__ void load_word_to_lds(const void *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}

// ROWS rows of D channels from memory to an LDS tile, in chunks of 16 bytes; the
// channels are `first` of one tensor, then `second` of another.  Rows behind the
// last (n - 1) repeat it; channels behind both are the row's first again: what
// they meet is 0, or their results are not kept.
template <int D, int ROWS, int THREADS, typename PERM> struct TileLoader {
    static constexpr int N = ROWS * D * 2 / 16 / THREADS;  // chunks a thread
    const char *base[N];
    uint32_t stride[N];
    __device__ __forceinline__ void init(const bf16_t *one, int64_t one_st, int first, const bf16_t *two, int64_t two_st, int second) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = i * THREADS + threadIdx.x, r = at / (D / 8);
            const int ch = (PERM::template place<D>(r, at % (D / 8)) - r * D * 2) / 2;
            const bool other = ch >= first && ch < first + second;
            base[i] = reinterpret_cast<const char *>(other ? two + (ch - first) : one + (ch < first ? ch : 0));
            stride[i] = static_cast<uint32_t>(other ? two_st : one_st) * 2;
        }
    }
    __device__ __forceinline__ void issue(int r0, int n, uint32_t to) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = (i * THREADS + threadIdx.x) / (D / 8);
            load_to_lds(base[i] + static_cast<uint64_t>(static_cast<uint32_t>(min(r0 + r, n - 1))) * stride[i], to + (i * THREADS + (threadIdx.x & ~63)) * 16);
        }
    }
};

// The wave's own side as operand: channels `first` from `one`, then `second` from
// `two` (the lane's row; a valid one also where `inside` is false), zeros elsewhere.
template <int D> __device__ __forceinline__ void load_own(bf16x8 (&f)[D / 16], const bf16_t *one, int first, const bf16_t *two, int second, bool inside, int h) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const int ch = 16 * s + 8 * h;
        const bool other = ch >= first && ch < first + second;
        frag8 v;
        v.u = *reinterpret_cast<const uint4 *>(other ? two + (ch - first) : one + (ch < first ? ch : 0));
        const uint32_t keep = inside && ch < first + second ? 0xffffffffu : 0u;
        v.u = make_uint4(v.u.x & keep, v.u.y & keep, v.u.z & keep, v.u.w & keep);
        f[s] = v.v;
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return static_cast<uint32_t>(f32_to_bf16(a)) | static_cast<uint32_t>(f32_to_bf16(b)) << 16;
}
// four values of a row, from a C tile's registers 4 i .. 4 i + 3
__device__ __forceinline__ void store4(bf16_t *to, const f32x16 &c, int i, float by) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(pack2(c[4 * i] * by, c[4 * i + 1] * by), pack2(c[4 * i + 2] * by, c[4 * i + 3] * by));
}
__device__ __forceinline__ void store4(float *to, const f32x16 &c, int i, float by) {
    *reinterpret_cast<f32x4 *>(to) = f32x4{c[4 * i] * by, c[4 * i + 1] * by, c[4 * i + 2] * by, c[4 * i + 3] * by};
}

}  // namespace kda
