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

// .. and PARTS operands that add up to them: what the first rounds off is the second
template <int PARTS> __device__ __forceinline__ void half_tile(bf16x8 (&f)[PARTS], const f32x16 &c, int s) {
    f[0] = half_tile(c, s);
    if constexpr (PARTS == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[1][i] = static_cast<__bf16>(c[8 * s + i] - static_cast<float>(f[0][i]));
    }
}
// acc += a (f[0] + ..)
template <int PARTS> __device__ __forceinline__ f32x16 mfma32(const bf16x8 &a, const bf16x8 (&f)[PARTS], f32x16 acc) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) acc = mfma32(a, f[i], acc);
    return acc;
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
// Read in both ways: s(r) has the row's low two bits above its third, so that 8
// rows' chunks differ for a read by rows and 4 rows' PAIRS of chunks for one by
// columns; 8 rows on, and for 128 channels the odd rows, which would lie on the
// even ones' banks, take other places again.
struct BothRead {
    template <int D> __device__ __forceinline__ static constexpr int turn(int r) {
        const int s = (((r & 3) << 1) | (r >> 2 & 1)) ^ ((r >> 3 & 1) << 1);
        return D == 128 ? s | (r & 1) << 3 : s;
    }
    template <int D> __device__ __forceinline__ static constexpr int place(int r, int c) { return r * (D * 2) + ((c ^ turn<D>(r)) * 16); }
    // A lane's place for the first 16 channels of row c32, by rows; k 16-channel steps further
    template <int D> __device__ __forceinline__ static uint32_t row(int lane) { return place<D>(lane & 31, lane >> 5); }
    template <int D> __device__ __forceinline__ static uint32_t step(uint32_t at, int k) {
        return D == 128 ? at ^ (32 * k) : (at ^ (32 * (k & 3))) + (k >> 2) * 128;
    }
    // .. and for 32 channels of 16 rows, by columns: rows 4 h + 0..3 and 8 rows on; block b of channels
    template <int D> __device__ __forceinline__ static uint32_t columns(int lane) {
        return place<D>(4 * (lane >> 5) + ((lane & 15) >> 2), 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) + 8 * (lane & 1);
    }
    template <int D> __device__ __forceinline__ static bf16x8 read_columns(const char *tile, uint32_t at, int b) {
        const char *from = D == 128 ? tile : tile + (b >> 1) * 128;
        const uint32_t turned = D == 128 ? at ^ (64 * b) : at ^ (64 * (b & 1));
        const uint2 lo = read_tr16(from + turned), hi = read_tr16(from + 8 * D * 2 + (turned ^ 32));
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
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory", "m0");
}
// .. from a base that all lanes share and 32-bit offsets
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(offset), "s"(base) : "memory", "m0");
}
// .. and 4 bytes a lane
__device__ __forceinline__ void load_word_to_lds(const void *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}

// Tile after tile of ROWS rows of D channels from memory to LDS, in chunks of 16
// bytes; the channels are `first` of one tensor, then, with TWO, `second` of another.  Rows
// behind the last (n - 1) repeat it; channels behind both are the row's first
// again: what they meet is 0, or their results are not kept.  The tensors' bases
// step in scalar registers, a lane's offsets inside a tile stay (in LDS where a
// kernel has no register for them: a spilled one's load would wait for the tile.
// The queries' gradient of 192 channels spills 8 registers all the same, which it
// reads where the last tile is not full, and 26, also in its products, with two parts);
// where the key has two parts, a chunk's lanes load from the one, then from the
// other.
template <int D, int ROWS, int THREADS, typename PERM, bool TWO, bool STORED = false> struct TileLoader {
    static constexpr int N = ROWS * D * 2 / 16 / THREADS;  // chunks a thread
    const char *one, *two;
    uint32_t one_st, two_st;  // bytes of a row
    uint32_t off[STORED ? 1 : N];
    uint32_t other;           // bit i: chunk i is of the second part
    uint32_t *s_off;          // STORED: the lanes' offsets in LDS, [N][THREADS]
    // from row r0 on
    __device__ __forceinline__ void init(const bf16_t *a, int64_t a_st, int first, const bf16_t *b, int64_t b_st, int second, int r0, uint32_t *s = nullptr) {
        s_off = s;
        one_st = static_cast<uint32_t>(a_st) * 2;
        two_st = static_cast<uint32_t>(b_st) * 2;
        one = reinterpret_cast<const char *>(a) + static_cast<uint64_t>(static_cast<uint32_t>(r0)) * one_st;
        two = reinterpret_cast<const char *>(b) + static_cast<uint64_t>(static_cast<uint32_t>(r0)) * two_st;
        other = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = i * THREADS + threadIdx.x, r = c / (D / 8);
            const int ch = (PERM::template place<D>(r, c % (D / 8)) - r * D * 2) / 2;
            const bool is = TWO && ch >= first && ch < first + second;
            const uint32_t at = r * (is ? two_st : one_st) + 2 * (is ? ch - first : ch < first ? ch : 0);
            if constexpr (STORED) s_off[i * THREADS + threadIdx.x] = at;
            else off[i] = at;
            other |= (is ? 1u : 0u) << i;
        }
    }
    __device__ __forceinline__ uint32_t offset(int i) const {
        if constexpr (STORED) return s_off[i * THREADS + threadIdx.x];
        else return off[i];
    }
    __device__ __forceinline__ void load(int i, uint32_t at, uint32_t to) const {
        to += i * THREADS * 16 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
        if (!TWO || !(other >> i & 1)) load_to_lds(one, at, to);
        if (TWO && (other >> i & 1)) load_to_lds(two, at, to);
    }
    __device__ __forceinline__ void issue(int r0, int n, uint32_t to) {
        if (r0 + ROWS <= n) {
#pragma unroll
            for (int i = 0; i < N; ++i) load(i, offset(i), to);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {  // the last tile
                const int r = (i * THREADS + threadIdx.x) / (D / 8), behind = max(0, r0 + r - (n - 1));
                load(i, offset(i) - static_cast<uint32_t>(behind) * (TWO && (other >> i & 1) ? two_st : one_st), to);
            }
        }
        one += static_cast<uint64_t>(one_st) * ROWS;
        if (TWO) two += static_cast<uint64_t>(two_st) * ROWS;
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
