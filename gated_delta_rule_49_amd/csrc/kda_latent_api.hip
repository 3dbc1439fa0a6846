// C ABI of latent attention, its positions and its cache (declared in
// include/kda.h): host-side validation, workspace sizing and dispatch.  No
// kernel is launched before every argument has been checked; nothing here
// allocates or synchronises.
#include "../../include/kda.h"
#include "kda_latent.hpp"

#include <initializer_list>

using namespace kda;

namespace {

constexpr int64_t kMost31 = (static_cast<int64_t>(1) << 31) - 1;
constexpr int64_t kMostRows = (static_cast<int64_t>(1) << 28) - 16;   // the gradients' (token, head) rows, in whole workgroups of 16: fewer than 2^32 threads
constexpr int64_t kMostTokens = (static_cast<int64_t>(1) << 26) - 4;  // appended tokens, in whole workgroups of 4

bool dtype_ok(int t) { return t == KDA_F32 || t == KDA_BF16; }
int64_t size_of(int t) { return t == KDA_F32 ? 4 : 2; }
bool flag_ok(int f) { return f == 0 || f == 1; }
bool misaligned(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 16) return true;
    return false;
}
// strides that rows of 16-byte vectors can have
kda_status check_strides(std::initializer_list<int64_t> strides) {
    for (const int64_t st : strides) {
        if (st < 0 || st > (static_cast<int64_t>(1) << 48)) return KDA_ERR_BAD_SHAPE;
        if (st % 8) return KDA_ERR_UNSUPPORTED;
    }
    return KDA_OK;
}
// whether [p, p + n) and [q, q + m) share a byte
bool overlap(const void *p, int64_t n, const void *q, int64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && n > 0 && m > 0 && a < b + static_cast<uintptr_t>(m) && b < a + static_cast<uintptr_t>(n);
}
// memory that a call reads, or writes
struct Span {
    const void *at;
    int64_t bytes;
};
// [B, T, H, d] with its strides, in elements of `size` bytes
Span span(const void *at, int64_t B, int64_t sb, int64_t T, int64_t st, int64_t H, int64_t sh, int64_t d, int64_t size) {
    if (!at || B == 0 || T == 0) return {nullptr, 0};
    return {at, ((B - 1) * sb + (T - 1) * st + (H - 1) * sh + d) * size};
}
Span dense(const void *at, int64_t n, int64_t size) { return {at, n * size}; }
// no output on an input or on another output
bool apart(std::initializer_list<Span> in, std::initializer_list<Span> out) {
    for (const Span *o = out.begin(); o != out.end(); ++o) {
        for (const Span &i : in)
            if (overlap(o->at, o->bytes, i.at, i.bytes)) return false;
        for (const Span *u = out.begin(); u != o; ++u)
            if (overlap(o->at, o->bytes, u->at, u->bytes)) return false;
    }
    return true;
}
// an axis of n elements, s apart
struct Axis {
    int64_t n, s;
};
// whether no two runs of d elements share memory: taken by size, each axis
// steps over all that the smaller ones reach
template <int N> bool distinct(Axis (&&ax)[N], int64_t d) {
    for (int i = 0; i < N; ++i)
        for (int j = i + 1; j < N; ++j)
            if (ax[j].s < ax[i].s) std::swap(ax[i], ax[j]);
    int64_t reach = d;
    for (const Axis &x : ax) {
        if (x.n <= 1) continue;
        if (x.s < reach) return false;
        reach += (x.n - 1) * x.s;
    }
    return true;
}
kda_status status_of(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

// -------------------------------------------------------------- rotary ----
// elements from the first to behind the last of a strided [B, T, H, D]
int64_t extent(const kda_rotary_args *a, int64_t sb, int64_t st, int64_t sh) {
    return (a->B - 1) * sb + (a->T - 1) * st + (a->H - 1) * sh + a->D;
}
kda_status rotary(const kda_rotary_args *a, bool back, void *hip_stream) {
    if (!a) return KDA_ERR_NULL_ARG;
    if (a->B < 0 || a->T < 0 || a->H < 1 || a->D < 1 || a->rotary_dim < 0 || a->rotary_dim % 2 || a->offset < 0 ||
        static_cast<int64_t>(a->offset) + a->rotary_dim > a->D)
        return KDA_ERR_BAD_SHAPE;
    if (!dtype_ok(a->dtype) || !flag_ok(a->interleaved) || a->D > 4096 || a->rotary_dim > 1024) return KDA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(a->B) * a->T > kMost31 || static_cast<int64_t>(a->H) * a->D > kMost31) return KDA_ERR_UNSUPPORTED;
    for (const int64_t st : {a->x_stride_b, a->x_stride_t, a->x_stride_h, a->out_stride_b, a->out_stride_t, a->out_stride_h})
        if (st < 0 || st > (static_cast<int64_t>(1) << 48)) return KDA_ERR_BAD_SHAPE;
    if (a->B == 0 || a->T == 0) return KDA_OK;
    if (!a->x || !a->out || (a->rotary_dim && !a->freqs)) return KDA_ERR_NULL_ARG;
    const int64_t e = size_of(a->dtype);
    if (reinterpret_cast<uintptr_t>(a->x) % e || reinterpret_cast<uintptr_t>(a->out) % e) return KDA_ERR_UNSUPPORTED;
    if (!distinct({{a->B, a->out_stride_b}, {a->T, a->out_stride_t}, {a->H, a->out_stride_h}}, a->D)) return KDA_ERR_BAD_SHAPE;
    const bool same = a->x == a->out && (a->B == 1 || a->x_stride_b == a->out_stride_b) && (a->T == 1 || a->x_stride_t == a->out_stride_t) &&
                      (a->H == 1 || a->x_stride_h == a->out_stride_h);
    if (!same && overlap(a->x, extent(a, a->x_stride_b, a->x_stride_t, a->x_stride_h) * e, a->out,
                         extent(a, a->out_stride_b, a->out_stride_t, a->out_stride_h) * e))
        return KDA_ERR_BAD_SHAPE;
    RotaryParams p{};
    p.x = a->x; p.out = a->out; p.pos = a->positions; p.freqs = a->freqs;
    p.x_sb = a->x_stride_b; p.x_st = a->x_stride_t; p.x_sh = a->x_stride_h;
    p.o_sb = a->out_stride_b; p.o_st = a->out_stride_t; p.o_sh = a->out_stride_h;
    p.p_sb = a->pos_stride_b; p.p_st = a->pos_stride_t;
    p.B = a->B; p.T = a->T; p.H = a->H; p.D = a->D; p.rot = a->rotary_dim; p.offset = a->offset;
    p.interleaved = a->interleaved; p.back = back; p.magnitude = a->magnitude;
    return status_of(launch_rotary(p, a->dtype, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------------------- prefill ----
kda_status check_prefill(const kda_latent_prefill_args *a, bool need_ptrs, bool need_out) {
    if (!a) return KDA_ERR_NULL_ARG;
    if (a->B < 1 || a->T < 0 || a->S < 0 || a->H < 1 || a->num_seqs < 0 || a->d_nope < 1 || a->d_rope < 0 || a->d_v < 1) return KDA_ERR_BAD_SHAPE;
    if (a->d_nope % 8 || a->d_rope % 8 || a->d_v % 8 || static_cast<int64_t>(a->d_nope) + a->d_rope > 192 || a->d_v > 128) return KDA_ERR_UNSUPPORTED;
    if (!dtype_ok(a->in_dtype) || !dtype_ok(a->out_dtype) || !flag_ok(a->causal) || !flag_ok(a->precise)) return KDA_ERR_UNSUPPORTED;
    if (!a->cu_seqlens_q != !a->cu_seqlens_k) return KDA_ERR_BAD_SHAPE;
    if (a->cu_seqlens_q ? a->B != 1 || a->num_seqs < 1 : a->num_seqs != a->B) return KDA_ERR_BAD_SHAPE;
    // a launch has fewer than 2^32 threads: up to 512 for a tile of 64 tokens or more (tiles of 16 are taken below
    // 2^16 tokens times heads only), 16 for each (token, head), one for four channels of dk_rope
    const int64_t tokens = static_cast<int64_t>(a->B) * std::max(a->T, a->S);
    if (static_cast<int64_t>(a->num_seqs) * a->H > (1 << 21) || a->num_seqs > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    if (tokens >= (1 << 28) || tokens * a->H >= (1 << 28) || tokens * a->d_rope >= (static_cast<int64_t>(1) << 33)) return KDA_ERR_UNSUPPORTED;
    const kda_status st = check_strides({a->q_stride_b, a->q_stride_t, a->q_stride_h, a->k_stride_b, a->k_stride_t, a->k_stride_h, a->r_stride_b,
                                         a->r_stride_t, a->v_stride_b, a->v_stride_t, a->v_stride_h});
    if (st != KDA_OK) return st;
    for (const int64_t t : {a->q_stride_t, a->k_stride_t, a->r_stride_t, a->v_stride_t, static_cast<int64_t>(a->H) * a->d_v})
        if (t >= (1 << 23)) return KDA_ERR_UNSUPPORTED;  // 32-bit offsets inside a tile
    if (!need_ptrs) return KDA_OK;
    if (a->T > 0 && (!a->q || (need_out && (!a->o || !a->lse)))) return KDA_ERR_NULL_ARG;
    if (a->S > 0 && (!a->k_nope || !a->v || (a->d_rope && !a->k_rope))) return KDA_ERR_NULL_ARG;
    if (misaligned({a->q, a->k_nope, a->k_rope, a->v, a->o})) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
struct Inputs {
    Span q, k, r, v, cu_q, cu_k;
};
Inputs inputs_of(const kda_latent_prefill_args *a) {
    const int64_t e = size_of(a->in_dtype);
    return {span(a->q, a->B, a->q_stride_b, a->T, a->q_stride_t, a->H, a->q_stride_h, a->d_nope + a->d_rope, e),
            span(a->k_nope, a->B, a->k_stride_b, a->S, a->k_stride_t, a->H, a->k_stride_h, a->d_nope, e),
            span(a->k_rope, a->B, a->r_stride_b, a->S, a->r_stride_t, 1, 0, a->d_rope, e),
            span(a->v, a->B, a->v_stride_b, a->S, a->v_stride_t, a->H, a->v_stride_h, a->d_v, e),
            dense(a->cu_seqlens_q, static_cast<int64_t>(a->num_seqs) + 1, 4), dense(a->cu_seqlens_k, static_cast<int64_t>(a->num_seqs) + 1, 4)};
}
LatentParams latent_params(const kda_latent_prefill_args *a) {
    LatentParams p{};
    p.q = a->q; p.kn = a->k_nope; p.kr = a->k_rope; p.v = a->v;
    p.q_sb = a->q_stride_b; p.q_st = a->q_stride_t; p.q_sh = a->q_stride_h;
    p.k_sb = a->k_stride_b; p.k_st = a->k_stride_t; p.k_sh = a->k_stride_h;
    p.r_sb = a->r_stride_b; p.r_st = a->r_stride_t;
    p.v_sb = a->v_stride_b; p.v_st = a->v_stride_t; p.v_sh = a->v_stride_h;
    p.cu_q = a->cu_seqlens_q; p.cu_k = a->cu_seqlens_k;
    p.o = a->o; p.lse = a->lse;
    p.B = a->B; p.T = a->T; p.S = a->S; p.H = a->H; p.dn = a->d_nope; p.dr = a->d_rope; p.dv = a->d_v; p.N = a->num_seqs;
    p.causal = a->causal; p.precise = a->precise; p.scale = a->scale;
    return p;
}
// status words, the table of the queries' tiles, of the keys' (gradients),
// then the gradients' fp32 buffers
struct Layout {
    LatentTiles q, k;
    size_t spill, entry_q, entry_k, stats, part, bytes;
};
Layout latent_layout(const kda_latent_prefill_args *a, bool grad) {
    Layout l{};
    const bool packed = a->cu_seqlens_q != nullptr;
    const int64_t queries = static_cast<int64_t>(a->B) * a->T, keys = static_cast<int64_t>(a->B) * a->S;
    l.q.size = grad ? latent_grad_tile_q(a->in_dtype, queries, a->H) : latent_tile_q(a->in_dtype, queries, a->H);
    l.k.size = latent_grad_tile_k(a->in_dtype, keys, a->H);
    l.q.bound = l.q.per_seq = latent_tiles_bound(a->T, a->num_seqs, l.q.size, packed);
    l.k.bound = l.k.per_seq = latent_tiles_bound(a->S, a->num_seqs, l.k.size, packed);
    l.spill = kAlign;
    l.entry_q = l.spill + (packed ? align_up(latent_table_spill(a->num_seqs)) : 0);
    l.entry_k = l.entry_q + (packed ? align_up(sizeof(int2) * l.q.bound) : 0);
    l.stats = l.entry_k + (packed && grad ? align_up(sizeof(int2) * l.k.bound) : 0);
    l.part = l.stats + (grad ? align_up(2 * sizeof(float) * a->B * a->T * a->H) : 0);
    l.bytes = l.part + (grad ? align_up(sizeof(float) * a->H * a->B * a->S * a->d_rope) : 0);
    return l;
}
// the table of packed sequences; unpacked calls have their status set
hipError_t prepare_tiles(const kda_latent_prefill_args *a, Layout &l, char *ws, bool grad, int32_t *user_status, hipStream_t s) {
    l.q.entry = reinterpret_cast<int2 *>(ws + l.entry_q);
    l.k.entry = reinterpret_cast<int2 *>(ws + l.entry_k);
    int32_t *word = reinterpret_cast<int32_t *>(ws);
    l.q.count = word + 1;
    l.k.count = word + 2;
    if (!a->cu_seqlens_q) return user_status ? launch_status_word(user_status, s) : hipSuccess;
    LatentTable t{};
    t.cu_q = a->cu_seqlens_q; t.cu_k = a->cu_seqlens_k;
    t.T = a->T; t.S = a->S; t.N = a->num_seqs;
    t.size_q = l.q.size;
    t.size_k = l.k.size;
    t.bound_q = l.q.bound;
    t.bound_k = l.k.bound;
    t.entry_q = reinterpret_cast<int2 *>(ws + l.entry_q);
    t.entry_k = grad ? reinterpret_cast<int2 *>(ws + l.entry_k) : nullptr;
    t.spill = reinterpret_cast<int32_t *>(ws + l.spill);
    t.causal = a->causal;
    t.word = word;
    t.user_status = user_status;
    return launch_latent_table(t, s);
}
// what the gradients read and write
struct GradSpans {
    Inputs in;
    Span o, lse, d_o, dq, dkn, dkr, dv, status;
};
GradSpans grad_spans(const kda_latent_backward_args *a) {
    const kda_latent_prefill_args &f = a->f;
    const int64_t e = size_of(f.in_dtype), queries = static_cast<int64_t>(f.B) * f.T * f.H, keys = static_cast<int64_t>(f.B) * f.S;
    return {inputs_of(&f),
            span(f.o, f.B, a->o_stride_b, f.T, a->o_stride_t, f.H, a->o_stride_h, f.d_v, size_of(f.out_dtype)),
            span(f.lse, f.B, a->lse_stride_b, f.T, a->lse_stride_t, f.H, a->lse_stride_h, 1, 4),
            span(a->d_o, f.B, a->d_o_stride_b, f.T, a->d_o_stride_t, f.H, a->d_o_stride_h, f.d_v, e),
            dense(a->dq, queries * (f.d_nope + f.d_rope), e), dense(a->dk_nope, keys * f.H * f.d_nope, e), dense(a->dk_rope, keys * f.d_rope, e),
            dense(a->dv, keys * f.H * f.d_v, e), dense(f.device_status, 1, 4)};
}
kda_status check_backward(const kda_latent_backward_args *a, bool need_ptrs) {
    if (!a) return KDA_ERR_NULL_ARG;
    kda_status st = check_prefill(&a->f, need_ptrs, true);
    if (st != KDA_OK) return st;
    st = check_strides({a->o_stride_b, a->o_stride_t, a->o_stride_h, a->d_o_stride_b, a->d_o_stride_t, a->d_o_stride_h});
    if (st != KDA_OK) return st;
    if (a->d_o_stride_t >= (1 << 23) || static_cast<int64_t>(a->f.B) * a->f.T * a->f.H > kMostRows) return KDA_ERR_UNSUPPORTED;
    for (const int64_t s : {a->lse_stride_b, a->lse_stride_t, a->lse_stride_h})
        if (s < 0 || s > (static_cast<int64_t>(1) << 48)) return KDA_ERR_BAD_SHAPE;
    if (!need_ptrs) return KDA_OK;
    if (a->f.T > 0 && (!a->d_o || !a->dq)) return KDA_ERR_NULL_ARG;
    if (a->f.S > 0 && (!a->dk_nope || !a->dv || (a->f.d_rope && !a->dk_rope))) return KDA_ERR_NULL_ARG;
    if (!a->f.d_rope && a->dk_rope) return KDA_ERR_BAD_SHAPE;
    if (misaligned({a->d_o, a->dq, a->dk_nope, a->dk_rope, a->dv})) return KDA_ERR_UNSUPPORTED;
    const GradSpans m = grad_spans(a);
    if (!apart({m.in.q, m.in.k, m.in.r, m.in.v, m.in.cu_q, m.in.cu_k, m.o, m.lse, m.d_o}, {m.dq, m.dkn, m.dkr, m.dv, m.status})) return KDA_ERR_BAD_SHAPE;
    return KDA_OK;
}

// -------------------------------------------------------------- decode ----
kda_status check_pages(int32_t num_pages, int32_t page_size, int32_t max_pages, int64_t page_stride, int64_t row_stride, int64_t table_stride, int64_t d) {
    if (num_pages < 1 || page_size < 1 || max_pages < 1 || table_stride < 0) return KDA_ERR_BAD_SHAPE;
    if (static_cast<int64_t>(max_pages) * page_size > kMost31 - 64) return KDA_ERR_UNSUPPORTED;  // rows of a last, partial step count in 32 bits
    const kda_status st = check_strides({page_stride, row_stride});
    if (st != KDA_OK) return st;
    // rows of one page, and one row of all pages, that do not share memory
    if ((page_size > 1 && row_stride < d) || (num_pages > 1 && page_stride < d)) return KDA_ERR_BAD_SHAPE;
    return KDA_OK;
}
struct DecodeSpans {
    Span q, cache, table, lengths, o, lse, status;
};
DecodeSpans decode_spans(const kda_latent_decode_args *a) {
    const int64_t e = size_of(a->in_dtype), d = a->d_latent + a->d_rope, rows = static_cast<int64_t>(a->B) * a->n_tokens * a->H;
    return {span(a->q, a->B, a->q_stride_b, a->n_tokens, a->q_stride_t, a->H, a->q_stride_h, d, e),
            span(a->cache, a->num_pages, a->page_stride, a->page_size, a->row_stride, 1, 0, d, e),
            span(a->page_table, a->B, a->table_stride, 1, 0, 1, 0, a->max_pages, 4), dense(a->lengths, a->B, 4),
            dense(a->o, rows * a->d_latent, size_of(a->out_dtype)), dense(a->lse, rows, 4), dense(a->device_status, 1, 4)};
}
kda_status check_decode(const kda_latent_decode_args *a, bool need_ptrs) {
    if (!a) return KDA_ERR_NULL_ARG;
    if (a->B < 0 || a->H < 1 || a->n_tokens < 1 || a->d_latent < 1 || a->d_rope < 0) return KDA_ERR_BAD_SHAPE;
    if (a->d_latent % 8 || a->d_rope % 8 || a->d_latent > 512 || static_cast<int64_t>(a->d_latent) + a->d_rope > 576) return KDA_ERR_UNSUPPORTED;
    if (!dtype_ok(a->in_dtype) || !dtype_ok(a->out_dtype)) return KDA_ERR_UNSUPPORTED;
    if (a->B > 65536 || static_cast<int64_t>(a->n_tokens) * a->H >= (1 << 24) || static_cast<int64_t>(a->B) * a->n_tokens * a->H >= (1 << 24))
        return KDA_ERR_UNSUPPORTED;
    kda_status st = check_pages(a->num_pages, a->page_size, a->max_pages, a->page_stride, a->row_stride, a->table_stride, a->d_latent + a->d_rope);
    if (st != KDA_OK) return st;
    st = check_strides({a->q_stride_b, a->q_stride_t, a->q_stride_h});
    if (st != KDA_OK) return st;
    if (!need_ptrs || a->B == 0) return KDA_OK;
    if (!a->q || !a->cache || !a->page_table || !a->lengths || !a->o || !a->lse) return KDA_ERR_NULL_ARG;
    if (misaligned({a->q, a->cache, a->o})) return KDA_ERR_UNSUPPORTED;
    const DecodeSpans m = decode_spans(a);
    if (!apart({m.q, m.cache, m.table, m.lengths}, {m.o, m.lse, m.status})) return KDA_ERR_BAD_SHAPE;
    return KDA_OK;
}
LatentDecodePlan decode_plan(const kda_latent_decode_args *a) {
    return latent_decode_plan(a->B, a->H, a->n_tokens, a->d_latent, a->d_rope, static_cast<int64_t>(a->max_pages) * a->page_size, a->in_dtype);
}

}  // namespace

extern "C" {

kda_status kda_rotary(const kda_rotary_args *a, void *hip_stream) { return rotary(a, false, hip_stream); }
kda_status kda_rotary_backward(const kda_rotary_args *a, void *hip_stream) { return rotary(a, true, hip_stream); }

kda_status kda_latent_append(const kda_latent_append_args *a, void *hip_stream) {
    if (!a) return KDA_ERR_NULL_ARG;
    if (a->B < 0 || a->T < 0 || a->num_seqs < 0 || a->d_latent < 1 || a->d_rope < 0) return KDA_ERR_BAD_SHAPE;
    if (a->d_latent % 8 || a->d_rope % 8 || a->d_latent > 2048 || a->d_rope > 256) return KDA_ERR_UNSUPPORTED;
    if (!dtype_ok(a->dtype) || !flag_ok(a->interleaved)) return KDA_ERR_UNSUPPORTED;
    if (!(a->eps >= 0.f)) return KDA_ERR_BAD_SHAPE;
    if (a->cu_seqlens ? a->B != 1 || a->num_seqs < 1 : a->num_seqs != a->B) return KDA_ERR_BAD_SHAPE;
    if (static_cast<int64_t>(a->B) * a->T > kMostTokens) return KDA_ERR_UNSUPPORTED;
    const int64_t d = a->d_latent + a->d_rope, e = size_of(a->dtype);
    kda_status st = check_pages(a->num_pages, a->page_size, a->max_pages, a->page_stride, a->row_stride, a->table_stride, d);
    if (st != KDA_OK) return st;
    // rows that are written, by a wave each, share no memory with any other
    if (!distinct({{a->num_pages, a->page_stride}, {a->page_size, a->row_stride}}, d)) return KDA_ERR_BAD_SHAPE;
    st = check_strides({a->kv_stride_b, a->kv_stride_t});
    if (st != KDA_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (a->B > 0 && a->T > 0) {
        if (!a->kv || !a->cache || !a->page_table || !a->lengths) return KDA_ERR_NULL_ARG;
        if (misaligned({a->kv, a->cache, a->rows})) return KDA_ERR_UNSUPPORTED;
        const int64_t kv = ((a->B - 1) * a->kv_stride_b + (a->T - 1) * a->kv_stride_t + d) * e;
        const int64_t cache = ((a->num_pages - 1) * a->page_stride + (a->page_size - 1) * a->row_stride + d) * e;
        const int64_t rows = static_cast<int64_t>(a->B) * a->T * d * e;
        if (overlap(a->kv, kv, a->cache, cache) || overlap(a->rows, rows, a->kv, kv) || overlap(a->rows, rows, a->cache, cache)) return KDA_ERR_BAD_SHAPE;
    }
    if (a->device_status && launch_status_word(a->device_status, s) != hipSuccess) return KDA_ERR_HIP;
    if (a->B == 0 || a->T == 0) return KDA_OK;
    LatentAppendParams p{};
    p.kv = a->kv; p.weight = a->norm_weight; p.freqs = a->freqs; p.cu = a->cu_seqlens; p.lengths = a->lengths; p.page_table = a->page_table;
    p.cache = a->cache; p.rows = a->rows; p.status = a->device_status;
    p.kv_sb = a->kv_stride_b; p.kv_st = a->kv_stride_t;
    p.page_stride = a->page_stride; p.row_stride = a->row_stride; p.table_stride = a->table_stride;
    p.B = a->B; p.T = a->T; p.N = a->num_seqs; p.dc = a->d_latent; p.dr = a->d_rope; p.interleaved = a->interleaved;
    p.num_pages = a->num_pages; p.page_size = a->page_size; p.max_pages = a->max_pages;
    p.eps = a->eps; p.magnitude = a->magnitude;
    return status_of(launch_latent_append(p, a->dtype, s));
}

size_t kda_latent_prefill_workspace_bytes(const kda_latent_prefill_args *a) {
    return check_prefill(a, false, false) == KDA_OK ? latent_layout(a, false).bytes : 0;
}

kda_status kda_latent_prefill(const kda_latent_prefill_args *a, void *hip_stream) {
    const kda_status st = check_prefill(a, true, true);
    if (st != KDA_OK) return st;
    const int64_t rows = static_cast<int64_t>(a->B) * a->T * a->H;
    const Inputs in = inputs_of(a);
    const Span o = dense(a->o, rows * a->d_v, size_of(a->out_dtype)), lse = dense(a->lse, rows, 4), status = dense(a->device_status, 1, 4);
    if (!apart({in.q, in.k, in.r, in.v, in.cu_q, in.cu_k}, {o, lse, status})) return KDA_ERR_BAD_SHAPE;
    if (!a->workspace) return KDA_ERR_NULL_ARG;
    if (reinterpret_cast<uintptr_t>(a->workspace) % kAlign) return KDA_ERR_BAD_SHAPE;
    Layout l = latent_layout(a, false);
    if (a->workspace_bytes < l.bytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
    const bool used = a->T > 0 || a->cu_seqlens_q;
    if (used && !apart({in.q, in.k, in.r, in.v, in.cu_q, in.cu_k, o, lse, status}, {dense(a->workspace, l.bytes, 1)})) return KDA_ERR_BAD_SHAPE;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    char *ws = static_cast<char *>(a->workspace);
    hipError_t e = prepare_tiles(a, l, ws, false, a->device_status, s);
    if (e != hipSuccess) return KDA_ERR_HIP;
    if (a->T == 0) return KDA_OK;
    LatentParams p = latent_params(a);
    p.tq = l.q;
    p.status = reinterpret_cast<int32_t *>(ws);
    return status_of(launch_latent_prefill(p, a->in_dtype, a->out_dtype, s));
}

size_t kda_latent_backward_workspace_bytes(const kda_latent_backward_args *a) {
    return check_backward(a, false) == KDA_OK ? latent_layout(&a->f, true).bytes : 0;
}

kda_status kda_latent_backward(const kda_latent_backward_args *a, void *hip_stream) {
    const kda_status st = check_backward(a, true);
    if (st != KDA_OK) return st;
    if (!a->workspace) return KDA_ERR_NULL_ARG;
    if (reinterpret_cast<uintptr_t>(a->workspace) % kAlign) return KDA_ERR_BAD_SHAPE;
    Layout l = latent_layout(&a->f, true);
    if (a->workspace_bytes < l.bytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
    const GradSpans m = grad_spans(a);
    if (!apart({m.in.q, m.in.k, m.in.r, m.in.v, m.in.cu_q, m.in.cu_k, m.o, m.lse, m.d_o, m.dq, m.dkn, m.dkr, m.dv, m.status}, {dense(a->workspace, l.bytes, 1)}))
        return KDA_ERR_BAD_SHAPE;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    char *ws = static_cast<char *>(a->workspace);
    hipError_t e = prepare_tiles(&a->f, l, ws, true, a->f.device_status, s);
    if (e != hipSuccess) return KDA_ERR_HIP;
    LatentGradParams g{};
    g.f = latent_params(&a->f);
    g.f.tq = l.q;
    g.f.status = reinterpret_cast<int32_t *>(ws);
    g.tk = l.k;
    g.d_o = a->d_o;
    g.o_dtype = a->f.out_dtype;
    g.dq = a->dq; g.dkn = a->dk_nope; g.dkr = a->dk_rope; g.dv = a->dv;
    g.o_sb = a->o_stride_b; g.o_st = a->o_stride_t; g.o_sh = a->o_stride_h;
    g.l_sb = a->lse_stride_b; g.l_st = a->lse_stride_t; g.l_sh = a->lse_stride_h;
    g.d_sb = a->d_o_stride_b; g.d_st = a->d_o_stride_t; g.d_sh = a->d_o_stride_h;
    g.lse2 = reinterpret_cast<float *>(ws + l.stats);
    g.delta = g.lse2 + static_cast<size_t>(a->f.B) * a->f.T * a->f.H;
    g.dkr_part = reinterpret_cast<float *>(ws + l.part);
    return status_of(launch_latent_backward(g, a->f.in_dtype, s));
}

size_t kda_latent_decode_workspace_bytes(const kda_latent_decode_args *a) {
    return check_decode(a, false) == KDA_OK ? decode_plan(a).bytes() + kAlign : 0;
}

kda_status kda_latent_decode(const kda_latent_decode_args *a, void *hip_stream) {
    const kda_status st = check_decode(a, true);
    if (st != KDA_OK) return st;
    if (!a->workspace) return KDA_ERR_NULL_ARG;
    if (reinterpret_cast<uintptr_t>(a->workspace) % kAlign) return KDA_ERR_BAD_SHAPE;
    const LatentDecodePlan plan = decode_plan(a);
    if (a->workspace_bytes < plan.bytes() + kAlign) return KDA_ERR_WORKSPACE_TOO_SMALL;
    const DecodeSpans m = decode_spans(a);
    if (a->B > 0 && !apart({m.q, m.cache, m.table, m.lengths, m.o, m.lse, m.status}, {dense(a->workspace, plan.bytes(), 1)})) return KDA_ERR_BAD_SHAPE;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (a->device_status && launch_status_word(a->device_status, s) != hipSuccess) return KDA_ERR_HIP;
    if (a->B == 0) return KDA_OK;
    LatentDecodeParams p{};
    p.q = a->q; p.cache = a->cache;
    p.q_sb = a->q_stride_b; p.q_st = a->q_stride_t; p.q_sh = a->q_stride_h;
    p.page_stride = a->page_stride; p.row_stride = a->row_stride; p.table_stride = a->table_stride;
    p.page_table = a->page_table; p.lengths = a->lengths;
    p.o = a->o; p.lse = a->lse; p.status = a->device_status;
    char *ws = static_cast<char *>(a->workspace);
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_lse = reinterpret_cast<float *>(ws + plan.o_bytes);
    p.info = reinterpret_cast<int2 *>(ws + plan.o_bytes + plan.lse_bytes);
    p.B = a->B; p.H = a->H; p.m = a->n_tokens; p.dc = a->d_latent; p.dr = a->d_rope;
    p.num_pages = a->num_pages; p.page_size = a->page_size; p.max_pages = a->max_pages;
    p.workers = plan.workers;
    // with 2^l the least power of 2 >= page_size and magic = ceil(2^(31 + l) / page_size): the product
    // exceeds k 2^(31 + l) / page_size by less than k 2^l <= 2^(31 + l), in units of 1 / page_size
    uint32_t l = 0;
    while ((static_cast<uint64_t>(1) << l) < static_cast<uint64_t>(a->page_size)) ++l;
    p.page_shift = 31 + l;
    p.page_magic = static_cast<uint32_t>(((static_cast<uint64_t>(1) << p.page_shift) + a->page_size - 1) / a->page_size);
    p.scale = a->scale;
    return status_of(launch_latent_decode(p, plan, a->in_dtype, a->out_dtype, s));
}

}  // extern "C"
