// Latent attention (expanded and absorbed forms), rotary positions and the
// paged latent cache: parameters and helpers that the kernels share.
#pragma once
#include "kda_launch.hpp"

namespace kda {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBadSeqlens = 6, kBadPages = 9;  // KDA_ERR_BAD_SEQLENS, KDA_ERR_BAD_PAGES

// ------------------------------------------------------------- expanded ----
// Work of the expanded form is cut into tiles of `size` tokens of one sequence
// (queries, or keys in the gradients).  Packed sequences: a table made on the
// device; else the place follows from the index.
struct LatentTiles {
    const int2 *entry;     // packed: (sequence, tile of it)
    const int32_t *count;  // packed: how many there are
    int32_t bound;         // tiles a head (an upper bound when packed)
    int32_t per_seq;       // unpacked: tiles of one sequence
    int32_t size;          // tokens of a tile
};
struct LatentParams {
    const void *q, *kn, *kr, *v;
    int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, r_sb, r_st, v_sb, v_st, v_sh;
    const int32_t *cu_q, *cu_k;  // packed, else null
    const int32_t *status;       // packed: 0 = offsets valid
    void *o;                     // [B, T, H, dv]
    float *lse;                  // [B, T, H]
    int32_t B, T, S, H, dn, dr, dv, N;
    int32_t causal, precise;
    float scale;
    LatentTiles tq;
};
struct LatentGradParams {
    LatentParams f;             // f.o, f.lse are read
    const void *d_o;
    int64_t o_sb, o_st, o_sh, l_sb, l_st, l_sh, d_sb, d_st, d_sh;  // strides of o, lse, d_o
    void *dq, *dkn, *dkr, *dv;
    float *lse2, *delta;        // [H, B T]: lse log2 e, rowsum(d_o o)
    float *dkr_part;            // [H, B S, dr]: each head's share of dk_rope
    LatentTiles tk;
    int32_t o_dtype;
};

// one (tile, head) of the grid
struct LatentPlace {
    int64_t q_row, k_row;  // the sequence's first row in [B T) and in [B S)
    int b, q0, k0;         // batch row; first query and key token in it
    int tq, tk;            // lengths
    int h, tile;
    bool valid;
};

// The tiles that see most come first, over all heads (`down`: the later ones), so
// that no long one begins late.  Blocks are dealt to the 8 XCDs in turn: where the
// heads divide evenly each XCD takes whole heads, whose keys and values are then
// read through one L2.
__device__ __forceinline__ LatentPlace latent_place(const LatentParams &p, const LatentTiles &t, int block, bool down) {
    LatentPlace a;
    const int pairs = p.cu_q ? p.H : p.H * p.N;
    const int per = p.cu_q ? t.bound : t.per_seq;
    int pair, i;
    if (pairs % 8 == 0) {
        i = (block >> 3) / (pairs / 8);
        pair = (block & 7) * (pairs / 8) + (block >> 3) - i * (pairs / 8);
    } else {
        i = block / pairs;
        pair = block - i * pairs;
    }
    if (p.cu_q) {
        const int n = *p.status == 0 ? *t.count : 0;
        a.valid = i < n;
        if (!a.valid) return a;
        const int2 e = t.entry[i];  // the largest first
        a.h = pair;
        a.b = 0;
        a.tile = e.y;
        a.q0 = p.cu_q[e.x];
        a.tq = p.cu_q[e.x + 1] - a.q0;
        a.k0 = p.cu_k[e.x];
        a.tk = p.cu_k[e.x + 1] - a.k0;
    } else {
        a.valid = true;
        a.b = pair / p.H;
        a.h = pair - a.b * p.H;
        a.tile = down ? per - 1 - i : i;
        a.q0 = a.k0 = 0;
        a.tq = p.T;
        a.tk = p.S;
    }
    // the same in all lanes, said so: the table's words come by vector loads
    for (int *x : {&a.b, &a.q0, &a.k0, &a.tq, &a.tk, &a.h, &a.tile}) *x = __builtin_amdgcn_readfirstlane(*x);
    a.q_row = static_cast<int64_t>(a.b) * p.T + a.q0;
    a.k_row = static_cast<int64_t>(a.b) * p.S + a.k0;
    return a;
}

// workspace of the expanded form: [0, 256) status and counts, then the tables
inline int latent_tiles_bound(int tokens, int seqs, int size, bool packed) {
    return packed ? (tokens + size - 1) / size + seqs : (tokens + size - 1) / size;
}
struct LatentTable {
    const int32_t *cu_q, *cu_k;
    int32_t T, S, N;
    int32_t size_q, size_k, bound_q, bound_k;
    int32_t causal;
    int2 *entry_q, *entry_k;    // entry_k null: queries only
    int32_t *spill;             // latent_table_spill(N) bytes
    int32_t *word;              // status, count of q tiles, count of k tiles
    int32_t *user_status;       // nullable
};
size_t latent_table_spill(int N);
hipError_t launch_latent_table(const LatentTable &t, hipStream_t s);
hipError_t launch_status_word(int32_t *word, hipStream_t s);  // *word = 0

// tokens of a query tile (forward, and the queries' gradient) and of a key
// tile (the keys' and values' gradient), by type and by how many tokens and heads there are
int latent_tile_q(int dtype, int64_t tokens, int H);
int latent_grad_tile_q(int dtype, int64_t tokens, int H);
int latent_grad_tile_k(int dtype, int64_t tokens, int H);
hipError_t launch_latent_prefill(const LatentParams &p, int in_dtype, int out_dtype, hipStream_t s);
hipError_t launch_latent_backward(const LatentGradParams &g, int in_dtype, hipStream_t s);
// the two types' own kernels
int latent_tile_f32(int64_t tokens, int H);
hipError_t latent_prefill_f32(const LatentParams &p, int out_dtype, hipStream_t s);
hipError_t latent_backward_f32(const LatentGradParams &g, hipStream_t s);

// ------------------------------------------------------------- absorbed ----
struct LatentDecodeParams {
    const void *q, *cache;
    int64_t q_sb, q_st, q_sh, page_stride, row_stride, table_stride;
    const int32_t *page_table, *lengths;
    void *o;
    float *lse;
    int32_t *status;       // nullable
    float *part_o;         // [row tiles, 2 workers, rows of a tile, dc]
    float *part_lse;       // [row tiles, 2 workers, rows of a tile]
    int2 *info;            // [B]: where a sequence's pieces are
    int32_t B, H, m, dc, dr;
    int32_t num_pages, page_size, max_pages;
    int32_t workers;       // workgroups a row tile is dealt to
    uint32_t page_magic, page_shift;  // k / page_size = k page_magic >> page_shift for k < 2^31
    float scale;
};
struct LatentDecodePlan {
    int32_t rows;      // rows (token, head) of a tile
    int32_t tiles;     // row tiles of a sequence
    int32_t workers;   // workgroups that each row tile's keys are dealt to
    size_t o_bytes, lse_bytes, info_bytes;
    size_t bytes() const { return o_bytes + lse_bytes + info_bytes; }
};
LatentDecodePlan latent_decode_plan(int B, int H, int m, int dc, int dr, int64_t most_rows, int in_dtype);
hipError_t launch_latent_decode(const LatentDecodeParams &p, const LatentDecodePlan &plan, int in_dtype, int out_dtype, hipStream_t s);

// ------------------------------------------------- positions, cache write ----
struct RotaryParams {
    const void *x;
    void *out;
    const int32_t *pos;    // nullable
    const double *freqs;
    int64_t x_sb, x_st, x_sh, o_sb, o_st, o_sh, p_sb, p_st;
    int64_t start;         // the launch's first token
    int32_t B, T, H, D, rot, offset, interleaved, back;
    float magnitude;
};
hipError_t launch_rotary(const RotaryParams &p, int dtype, hipStream_t s);
struct LatentAppendParams {
    const void *kv;
    const float *weight;   // nullable
    const double *freqs;   // nullable
    const int32_t *cu, *lengths, *page_table;  // cu nullable
    void *cache, *rows;    // rows nullable
    int32_t *status;       // nullable
    int64_t kv_sb, kv_st, page_stride, row_stride, table_stride;
    int32_t B, T, N, dc, dr, interleaved;
    int32_t num_pages, page_size, max_pages;
    float eps, magnitude;
};
hipError_t launch_latent_append(const LatentAppendParams &p, int dtype, hipStream_t s);

// ---------------------------------------------------------------- device ----
// The sine and cosine of p f: the angle and its distance from the nearest
// multiple of pi / 2 in 64 bits, |r| <= pi / 4, then their Taylor series in
// fp32 (first terms left out: r^11 / 11! and r^12 / 12! < 2e-9 of the value).
__device__ __forceinline__ void sincos_far(double angle, float &sn, float &cs) {
    constexpr double kTwoOverPi = 0.63661977236758134308;
    constexpr double kPiHalf = 1.57079632679489655800, kPiHalfLo = 6.12323399573676603587e-17;
    const double n = rint(angle * kTwoOverPi);
    const float r = static_cast<float>(fma(-n, kPiHalfLo, fma(-n, kPiHalf, angle)));
    const int quarter = static_cast<int>(static_cast<int64_t>(n)) & 3;
    const float q = r * r;
    float a = 1.f / 362880.f;
    a = fmaf(a, q, -1.f / 5040.f);
    a = fmaf(a, q, 1.f / 120.f);
    a = fmaf(a, q, -1.f / 6.f);
    const float s = fmaf(r * q, a, r);
    float b = -1.f / 3628800.f;
    b = fmaf(b, q, 1.f / 40320.f);
    b = fmaf(b, q, -1.f / 720.f);
    b = fmaf(b, q, 1.f / 24.f);
    b = fmaf(b, q, -0.5f);
    const float c = fmaf(q, b, 1.f);
    sn = quarter & 1 ? c : s;
    cs = quarter & 1 ? s : c;
    if (quarter & 2) sn = -sn;
    if ((quarter + 1) & 2) cs = -cs;
}

}  // namespace kda
