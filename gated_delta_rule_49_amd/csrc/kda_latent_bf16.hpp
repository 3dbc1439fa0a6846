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
// A tile that is read in both ways uses the first permutation; see there.
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

// byte offset of chunk c of row r of a tile read by rows
template <int D> __device__ __forceinline__ constexpr int row_chunk(int r, int c) {
    if constexpr (D == 128) return r * (D * 2) + ((c ^ (r & 15)) * 16);
    else return r * (D * 2) + ((c & ~7) * 16) + (((c ^ r ^ (r >> 3 & 1)) & 7) * 16);
}
// .. and of a tile read by columns
template <int D> __device__ __forceinline__ constexpr int col_chunk(int r, int c) {
    const int t = r & 3;
    if constexpr (D == 64) return r * (D * 2) + ((c ^ (t << 1)) * 16);
    else return r * (D * 2) + ((c ^ (((t << 1) ^ ((t ^ (t >> 1)) & 1)) << 1)) * 16);
}

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

}  // namespace kda
