// Selective state space scan in chunked form: shared by the prompt scan
// (kda_ssm_prefill.hpp) and the gradients (kda_ssm_backward.hpp); the step sizes'
// softplus is the token step's too (kda_ssm_decode.hip).
//
// Over a chunk of L tokens, with la_t = A dt_t (all logs base 2 in the code),
// suf_t = sum_{s > t} la_s, tot = sum la, w_t = dt_t 2^suf_t:
//     S_out = 2^tot S_in + sum_t B_t (w_t x_t)^T
//     y_t   = 2^(-suf_t) [ C_t^T (2^tot S_in) + sum_{s <= t} (C_t . B_s) w_s x_s ] + D x_t
// The causal scores C_t . B_s do not depend on the head: a workgroup whose
// waves own heads of one group computes them once, and per head only the row
// factors 2^(-suf_t) and the scaled inputs w_t x_t are left.  That form is
// exact while 2^tot stays a normal number with room for its low-order parts;
// a chunk that decays by more than kFastTot takes the second form,
//     y_t = 2^(cum_t) C_t^T S_in + sum_{s <= t} (C_t . B_s) 2^(suf_s - suf_t) dt_s x_s ,
// every exponent <= 0.  suf_s - suf_t may be one token's small log beside sums of
// thousands (steps of mixed sizes in one head): where y is made the sums are in 64
// bits, kept as two floats for the second form.
//
// Precision: bf16 inputs enter the matrix cores as they are.  An fp32 operand is
// split into bf16 parts, every part but the last cut off or rounded: two hold it
// to 2^-15, three hold all 24 bits.  fp32 inputs take three; so does w x, which
// makes the state; the scores and the state behind y as many as y's type needs
// (ScanCfg), the operands of the gradients as theirs (GradCfg).  Products of two
// later parts, below 2^-14 (2 parts) or 2^-20 (3) of the term, are left out.
// Everything accumulates in fp32.
#pragma once
#include "kda_launch.hpp"

namespace kda {

// log(1 + e^x) to a few 2^-24 of ITSELF (softplus_f32 is so only in absolute
// terms): step sizes of 0.001 multiply logs that add up over a long memory.
//   e^-|x| = 2^n 2^r with n = rint(-|x| log2 e), r by a fused multiply-add
//            against both halves of log2 e, |r| <= 1/2
//   log(1 + y) = 2 atanh(y / (2 + y)), |y / (2 + y)| <= 1/3: seven odd terms
//            leave less than (1/9)^7 / 15 = 1.4e-8 of it
// e^-200 is below the smallest float, so |x| counts no further than 200: r would
// not stay small, and a step masked by the lowest value or -inf (a step of 0)
// would become NaN.
__device__ __forceinline__ float softplus_rel(float x) {
    constexpr float kLog2eLo = 1.92596299e-08f;  // log2 e - kLog2e
    const float m = fmaxf(-fabsf(x), -200.f);
    const float n = rintf(m * kLog2e);
    const float r = fmaf(m, kLog2eLo, fmaf(m, kLog2e, -n));
    const float y = ldexpf(fast_exp2(r), static_cast<int>(n));
    const float s = y / (2.f + y), q = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    const float l = 2.f * fmaf(s * q, p, s);
    return x != x ? x : fmaxf(x, 0.f) + l;
}

// A chunk whose total decay is above 2^-kFastTot may use the first form.  The
// state's own scale puts the chunk's factors around 1: from 2^(-kFastTot / 2) to
// 2^(kFastTot / 2) for w, the inverse for the rows.  Low-order parts reach down
// to about 2^(-kFastTot / 2 - 24), far above the smallest normal number 2^-126,
// and values below 2^64 do not overflow.  (With the scale fixed at the chunk's
// end the limit is 56: heads of A = -16 and steps of 0.1 pass it by far, and 32768
// tokens of 64 such heads take 395 us in phase 2, 329 to 354 so; inputs
// without wide decays take 315 to 330.)
constexpr float kFastTot = 112.f;
// A token whose own log is below this ends everything before it: 2^-256 is 0 in
// fp32 whatever it multiplies.  The log is taken as -256 then, so that sums over a
// chunk keep the small logs beside it.
constexpr float kGone = -256.f;
// how far a kept state's scale may go from 1 (log2) before it is multiplied out
constexpr double kLevel = 24.0;

struct SsmScan {
    SsmParams p;
    const int32_t *seg_off;   // packed: [N + 1] first segment of each sequence
    const int4 *seg_info;     // packed: (first token, length, sequence, index in its sequence)
    const int32_t *chunk_off; // packed: [N + 1] first chunk of each sequence
    const int32_t *status;    // packed: 0 = offsets valid
    int32_t *user_status;     // nullable
    float *seg_state;         // [segments, H, Ns, P]: the state entering each (phase 1: its own end state); null = unsplit
    float *seg_log;           // [segments, H]: log2 of each segment's decay
    int32_t seg_chunks;       // chunks of KDA_SSM_CHUNK tokens per segment
    int32_t segs_bound;       // grid bound on the number of segments
    int32_t segs_per_seq;     // unpacked
    int32_t chunks_per_seq;   // ceil(T / 64)
    int32_t state_chunk;      // tokens between the chunk_states written: 64, or 32 (fp32 gradients)
};

struct SsmSeg {
    int row, t0, len, n, s, count;  // batch row, first token of it, tokens, sequence, index, segments of the sequence
    int chunk;                      // first chunk's index among all chunks
    bool valid;
};
__device__ __forceinline__ SsmSeg ssm_seg(const SsmScan &q, int x) {
    SsmSeg g;
    if (q.p.cu_seqlens) {
        g.valid = *q.status == 0 && x < q.seg_off[q.p.N];
        if (!g.valid) return g;
        const int4 i = q.seg_info[x];
        g.row = 0; g.t0 = i.x; g.len = i.y; g.n = i.z; g.s = i.w;
        g.count = q.seg_off[g.n + 1] - q.seg_off[g.n];
        g.chunk = q.chunk_off[g.n] + g.s * q.seg_chunks;
    } else {
        g.valid = x < q.p.N * q.segs_per_seq;
        g.n = x / q.segs_per_seq;
        g.s = x % q.segs_per_seq;
        g.row = g.n;
        g.t0 = g.s * q.seg_chunks * 64;
        g.len = min(q.p.T - g.t0, q.seg_chunks * 64);
        g.count = q.segs_per_seq;
        g.chunk = g.n * q.chunks_per_seq + g.s * q.seg_chunks;
    }
    return g;
}

// Blocks of one segment and group are neighbours in the logical order; the
// hardware deals consecutive block numbers to the 8 XCDs in turn, so each XCD
// takes a contiguous run of the logical order and shares B and C in its L2.
__device__ __forceinline__ int xcd_order(int block, int grid) { return (block & 7) * (grid >> 3) + (block >> 3); }

// ---------------------------------------------------------------- operands --
// NPART bf16 parts of 8 values
template <int N> struct parts8 { frag8 f[N]; };

template <int N>
__device__ __forceinline__ void split_to(parts8<N> &o, int slot, float v) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bf16_t h = f32_to_bf16(v);
        o.f[i].s[slot] = h;
        if (i + 1 < N) v -= bf16_to_f32(h);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // one v_cvt_pk_bf16_f32
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
// Two neighbouring slots at once.  Every part but the last is the value's
// upper half as it stands (8 significant bits: three parts hold all 24), which
// one byte permutation packs and one mask and subtraction take off; the last
// is rounded.  (v_dot2c_f32_bf16 would take a part off in one instruction, but
// issues at a quarter of the rate: 1470 cycles against 960 for a wave's 32 x 64
// values.)
template <int N>
__device__ __forceinline__ void split_pair(parts8<N> &o, int slot, float v0, float v1) {
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) {
        const uint32_t u0 = __float_as_uint(v0), u1 = __float_as_uint(v1);
        o.f[i].w[slot / 2] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
        v0 -= __uint_as_float(u0 & 0xffff0000u);
        v1 -= __uint_as_float(u1 & 0xffff0000u);
    }
    o.f[N - 1].w[slot / 2] = pack_bf16(v0, v1);
}

// base (uniform) plus a lane's offset in elements, as a 32-bit byte offset.
// The empty statement keeps the base in scalar registers: rows a stride apart
// would otherwise become a chain of 64-bit vector additions.
template <typename T>
__device__ __forceinline__ T *lane_at(T *base, uint32_t elements) {
    typedef __attribute__((address_space(1))) char global_char;
    uint64_t at = reinterpret_cast<uint64_t>(base);
    asm("" : "+s"(at));
    return (T *)((global_char *)at + elements * static_cast<uint32_t>(sizeof(T)));
}

// c += A B over the parts' products whose orders add up to less than ORD
template <int NA, int NB, int ORD>
__device__ __forceinline__ void mfma_parts(f32x4 &c, const parts8<NA> &a, const parts8<NB> &b) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j < ORD) c = mfma16(a.f[i].v, b.f[j].v, c);
}

// the same for CT neighbouring tiles, the tiles innermost: consecutive
// instructions then accumulate into different registers
template <int NA, int NB, int ORD, int CT>
__device__ __forceinline__ void mfma_tiles(f32x4 (&c)[CT], const parts8<NA> &a, const parts8<NB> (&b)[CT]) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j < ORD)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) c[ct] = mfma16(a.f[i].v, b[ct].f[j].v, c[ct]);
}

// Position of the 4-element granule q of a 32-column step: an operand's lane
// group g = l / 16 reads granules g and 4 + g (kperm's slots) as one 16-byte
// piece.
__device__ __forceinline__ constexpr int granule_pos(int q) { return q < 4 ? 2 * q : 2 * (q - 4) + 1; }
// element offset of column k (a multiple of 4) in a row of 32-column steps
__device__ __forceinline__ constexpr int col_pos(int k) { return (k & ~31) + granule_pos((k >> 2) & 7) * 4; }

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

// Operand with its contraction along the rows [r0, r0 + 32) of a granule-
// ordered LDS tile and its 16 columns from c0 (ds_read_b64_tr_b16: lane i of
// group g addresses four columns of row r0 + 4 g + i / 4 and receives column
// c0 + i of rows r0 + 4 g + 0..3).
__device__ __forceinline__ void load_cols(frag8 &f, const bf16_t *tile, int stride, int r0, int c0, int g, int c16) {
    const bf16_t *at = tile + (r0 + 4 * g + (c16 >> 2)) * stride + col_pos(c0 + 4 * (c16 & 3));
    const v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(at));
    const v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(at + 16 * stride));
    const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
    f.u = make_uint4(ua.x, ua.y, ub.x, ub.y);
}
// Operand with its contraction along a row: rows [r0, r0 + 16), step kk
__device__ __forceinline__ void load_rows(frag8 &f, const bf16_t *tile, int stride, int r0, int kk, int g, int c16) {
    f.u = *reinterpret_cast<const uint4 *>(tile + (r0 + c16) * stride + kk * 32 + 8 * g);
}

union granule {
    bf16_t s[4];
    uint2 u;
};

// Four tokens by four channels of B or C as loaded
template <typename T> struct quad;
template <> struct quad<bf16_t> {
    uint2 r[4];
    static constexpr int PARTS = 1;
    __device__ __forceinline__ void ld(int i, const bf16_t *p) { r[i] = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void zero(int i) { r[i] = make_uint2(0, 0); }
    // part `part` of the four channels of token i
    __device__ __forceinline__ granule row(int i, int) const { granule g; g.u = r[i]; return g; }
};
template <> struct quad<float> {
    f32x4 r[4];
    static constexpr int PARTS = 3;
    __device__ __forceinline__ void ld(int i, const float *p) { r[i] = *reinterpret_cast<const f32x4 *>(p); }
    __device__ __forceinline__ void zero(int i) { r[i] = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ static bf16_t part_of(float v, int part) {
        for (int k = 0; k < part; ++k) v -= bf16_to_f32(f32_to_bf16(v));
        return f32_to_bf16(v);
    }
    __device__ __forceinline__ granule row(int i, int part) const {
        granule g;
#pragma unroll
        for (int c = 0; c < 4; ++c) g.s[c] = part_of(r[i][c], part);
        return g;
    }
};

// PW / 16 neighbouring channels of one token, as a lane loads and stores them
template <typename T, int CT> struct lanevec;
template <> struct lanevec<bf16_t, 1> {
    bf16_t u;
    __device__ __forceinline__ void ld(const bf16_t *p) { u = *p; }
    __device__ __forceinline__ float get(int) const { return bf16_to_f32(u); }
    __device__ __forceinline__ static void st(bf16_t *p, const float (&v)[1]) { *p = f32_to_bf16(v[0]); }
};
template <> struct lanevec<bf16_t, 2> {
    uint32_t u;
    __device__ __forceinline__ void ld(const bf16_t *p) { u = *reinterpret_cast<const uint32_t *>(p); }
    __device__ __forceinline__ float get(int c) const { return __uint_as_float(c ? (u & 0xffff0000u) : (u << 16)); }
    __device__ __forceinline__ static void st(bf16_t *p, const float (&v)[2]) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16(v[0], v[1]);
    }
};
template <> struct lanevec<float, 1> {
    float u;
    __device__ __forceinline__ void ld(const float *p) { u = *p; }
    __device__ __forceinline__ float get(int) const { return u; }
    __device__ __forceinline__ static void st(float *p, const float (&v)[1]) { *p = v[0]; }
};
template <> struct lanevec<float, 2> {
    float2 u;
    __device__ __forceinline__ void ld(const float *p) { u = *reinterpret_cast<const float2 *>(p); }
    __device__ __forceinline__ float get(int c) const { return c ? u.y : u.x; }
    __device__ __forceinline__ static void st(float *p, const float (&v)[2]) { *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]); }
};

// A wave's exchange with itself through LDS: its own writes before its reads.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Inclusive sums over the lanes up to each, without LDS: within rows of 16
// lanes (row_shr), then each row's and each half's last value to the lanes
// above (row_bcast:15, row_bcast:31).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, true));
}
// the same of both halves of a 64-bit value
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_moved(double v) {
    const int2 x = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, x.x, CTRL, ROWS, 0xf, true),
                                                __builtin_amdgcn_update_dpp(0, x.y, CTRL, ROWS, 0xf, true)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) { return v + dpp_moved<CTRL, ROWS>(v); }
template <typename T>
__device__ __forceinline__ T lane_scan(T v) {
    v = dpp_add<0x111, 0xf>(v);  // row_shr:1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
    return v;
}
// the value of the lane below, 0 for lane 0
__device__ __forceinline__ float lane_shift(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x138, 0xf, 0xf, true));  // wave_shr:1
}
__device__ __forceinline__ double lane_shift(double v) { return dpp_moved<0x138, 0xf>(v); }
// the last lane's value, uniform
__device__ __forceinline__ float last_lane(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
    const int2 x = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(x.x, 63), __builtin_amdgcn_readlane(x.y, 63)));
}

// Workspace layout, the tables of packed sequences and how a scan is split
// (host).  bytes: of the whole layout; the state and log arrays are there
// only where the scan may be split.
struct SsmPlan {
    int32_t seg_chunks, segs_bound, segs_per_seq, chunks_per_seq;
    int64_t chunks_bound;
    int32_t waves, blocks_per_group;  // of a workgroup; workgroups per segment and group
    bool split;
    size_t table_bytes, state_bytes, log_bytes;
    size_t bytes() const { return table_bytes + state_bytes + log_bytes; }
};
// walks: 1, or 2 for a pass from both ends at once
SsmPlan ssm_plan(const SsmParams &p, bool packed, int walks);
// fills the tables' pointers of q from a workspace laid out by the plan
void ssm_layout(SsmScan &q, const SsmPlan &plan, char *ws);

// segment and chunk tables of packed sequences; checks the offsets
hipError_t launch_ssm_table(const SsmScan &q, hipStream_t s);
// one phase of a scan; FULL writes y, the others only states.  phase 1: from
// zero, the end state and log decay of every segment but the last (reverse:
// but the first); phase 2: from the entering states.
enum { SSM_FULL = 0, SSM_STATES = 1, SSM_REVERSE = 2 };
hipError_t launch_ssm_phase(const SsmScan &q, const SsmPlan &plan, int phase, int in_dtype, int out_dtype, hipStream_t s);
hipError_t launch_ssm_states(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int phase, int in_dtype, hipStream_t s);
// Gradients (kda_ssm_backward.hpp)
struct SsmGrad {
    SsmScan q;                  // p.x, p.Bm, p.Cm, p.dt as in the forward
    const void *d_y;            // [B, T, H, P]
    const float *states, *gstates;  // [chunks * SUB, H, Ns, P]: entering each chunk, from the left / from the right
    void *dx, *ddt, *dB, *dC;
    float *part_B, *part_C;     // [splits, B T, G, Ns] where a group's heads are split, else null
    float *scalars;             // [3, H, items]: dA, dD, ddt_bias of every chunk
    int32_t heads_per_block, splits;
};
hipError_t ssm_grad_bf16(const SsmGrad &a, hipStream_t s);
hipError_t ssm_grad_f32(const SsmGrad &a, hipStream_t s);
// all of a backward pass; the workspace's layout is the plan's
struct SsmGradPlan {
    SsmPlan scan;
    int32_t sub, splits, heads_per_block;
    int64_t items;  // bound on the chunks (parts of 64 tokens in fp32)
    size_t state_bytes, part_bytes, scalar_bytes;
    size_t bytes() const { return scan.bytes() + scan.state_bytes + scan.log_bytes + 2 * state_bytes + 2 * part_bytes + scalar_bytes; }
};
SsmGradPlan ssm_grad_plan(const SsmParams &p, bool packed, int in_dtype);
struct SsmGradOut {
    const void *d_y;
    const float *d_final;
    void *dx, *ddt, *dB, *dC;
    float *dA, *dD, *ddt_bias, *d_initial;
};
hipError_t launch_ssm_backward(const SsmParams &p, const SsmGradOut &o, char *ws, int in_dtype, hipStream_t s);
// a whole scan: phases and the chain of segments between them
hipError_t launch_ssm_scan(const SsmScan &q, const SsmPlan &plan, int in_dtype, int out_dtype, hipStream_t s);
// the states alone, f from the left and r from the right (with segment states
// of its own), side by side
hipError_t launch_ssm_both(const SsmScan &f, const SsmScan &r, const SsmPlan &plan, int in_dtype, hipStream_t s);

}  // namespace kda
