// Latent attention's absorbed form on the bf16 matrix cores.
//
// A workgroup of eight waves takes 32 rows (token, head) of a sequence and a run
// of the cache, 64 rows (keys) a step, which come from memory to LDS directly, one
// step ahead: 74 KB in flight on every CU.  A step's rows are read twice, by rows
// as keys and by columns as values.
//   S^T = K Q^T    wave w: keys 16 (w % 4), rows 16 (w / 4), all channels
//                  (16 x 16 x 32 products; Q stays in registers)
//   P              to LDS, as two bf16 parts, over a maximum that all waves know
//   O^T += C^T P^T wave w: an eighth of the latent channels, all rows
//                  (32 x 32 x 16 products, one for each part of P)
// One part of P would leave each term of a sum off by up to 2^-8 of itself, and
// sums whose terms cancel by several of their own steps, an fp32 o too; it saves
// little where memory bounds: 235 us for 237 with two, 259 for 280 in the
// second case below.
// The maximum moves when some wave's scores pass it by more than kSlack, which
// the waves see together after the barrier that P needs anyway; then P is made
// again.  So a step takes two barriers, a moving maximum a third.
//
// More than 32 rows take more workgroups over the same keys, on the same XCD: its
// L2 then serves all but the first.  (64 rows a workgroup need 208 registers a
// lane for Q and the result alone; with what the loop keeps besides they spill,
// and a spilled value's load waits for the rows in flight: 12 rows of 64 heads
// over 280000 keys took 602 us so, 372 with 32 rows.)
//
// 128 sequences of up to 16384 rows, one token of 32 heads: 237 us with the join,
// 5.06 TB/s, bound by memory.  3 sequences of up to 131072, 4 tokens of 64 heads:
// 280 us, bound by the stages of a step, which follow each other (4200 cycles, 1150
// of them the CU's 64 bytes a cycle from L2).
#include "kda_latent_bf16.hpp"
#include "kda_latent_decode.hpp"

namespace kda {

namespace {

constexpr int kKeys = 64, kRows = 32, kThreads = 512;
constexpr float kSlack = 8.f;          // log2; see the forward: how far P may pass 1
constexpr int kPRow = kKeys * 2 + 16;  // bytes of a row of P: 16 more than its keys
constexpr int kPPart = kRows * kPRow;  // .. and of one part of it

// where chunk c of row r of the tile lies in its row (read by rows and by columns)
__device__ __forceinline__ constexpr int swizzle(int r, int c) { return c ^ BothRead::turn<0>(r); }

template <int DK> struct Shared {
    // the small parts first: their addresses are immediates of the instructions
    float most[4][kRows];    // each 16 keys' maximum
    float sum[4][kRows];
    const char *row[2][kKeys];
    int32_t page[2][kKeys];
    DecodeShared<kThreads> run;
    char p[2 * kPPart];
    __attribute__((aligned(128))) char tile[2][kKeys * DK * 2];
};

// The same value, computed where it stands: what follows from it is not kept in
// registers over the loop before.
__device__ __forceinline__ int here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}
__device__ __forceinline__ float quarters_max(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return swap_halves_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
template <typename O, int DK, int DC>
__global__ void __launch_bounds__(kThreads, 1) decode_bf16_kernel(LatentDecodeParams p, int tiles) {
    constexpr int NC = kKeys * DK / 8 / kThreads;      // chunks a thread
    constexpr int NB = DC / 256 ? DC / 256 : 1;        // 32-channel blocks a wave
    __shared__ __attribute__((aligned(128))) Shared<DK> sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c16 = lane & 15, h2 = lane >> 5, c32 = lane & 31;
    const int kg = wave & 3, own = (wave >> 2) * 16 + c16;  // the wave's keys, the lane's row of S^T
    int tile, worker;
    if (p.workers % 8 == 0) {  // the row tiles of one worker on one XCD
        const int x = blockIdx.x >> 3;
        tile = x % tiles;
        worker = (x / tiles) * 8 + (blockIdx.x & 7);
    } else {
        tile = blockIdx.x % tiles;
        worker = blockIdx.x / tiles;
    }
    DecodeRun run = decode_run<kThreads, kKeys>(p, worker, sh.run);
    const int d = p.dc + p.dr, rows = p.m * p.H;
    // scores are masked before they are scaled: the scale's sign goes to the query
    const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e;
    const uint32_t sign = p.scale < 0.f ? 0x80008000u : 0u;

    uint32_t chunk[NC];  // (row of the tile, byte of its channels) of the thread's chunks
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int at = i * kThreads + tid, r = at / (DK / 8), ch = swizzle(r, at % (DK / 8)) * 8;
        chunk[i] = static_cast<uint32_t>(r) << 16 | static_cast<uint32_t>(ch < d ? ch * 2 : 0);  // channels behind the last meet zeros of q
    }
    const uint32_t lds = lds_address(sh.tile[0]), pages = lds_address(sh.page[0]);
    // the lane's bytes in a tile: its key's row, chunk g (bit 2 of the chunk is the step's parity)
    const uint32_t key_at = static_cast<uint32_t>(kg * 16 + c16) * (DK * 2) + swizzle(c16, g) * 16;
    // .. and its four channels of row c16 / 4 of a half's eight (rows 4 further: bit 0 of the chunk turns)
    const uint32_t value_at = static_cast<uint32_t>(8 * h2 + (c16 >> 2)) * (DK * 2) + swizzle(8 * h2 + (c16 >> 2), 2 * (g & 1) + ((c16 & 3) >> 1)) * 16 + 8 * (c16 & 1);

    bool first = true;
    while (run.left > 0) {
        const int n = decode_rows(p, run.b);
        const int64_t steps = (n + kKeys - 1) / kKeys;
        if (steps == 0) { ++run.b; continue; }
        const int s0 = first ? static_cast<int>(run.at - run.before) : 0;
        const int count = static_cast<int>(min(run.left, steps - s0));
        if (s0 == 0 && tile == 0 && tid == 0) p.info[run.b] = decode_info(first, run.per, run.before, steps, worker);

        // The place of row `lane` of step i (a row behind the last stands for the step's first: its weight is 0).
        // Its page comes two steps ahead by the same way as the rows: a load that the compiler
        // knows would be waited for together with the rows in flight.
        const int32_t *table = p.page_table + run.b * p.table_stride;
        bool bad = p.lengths[run.b] != n;
        auto key_of = [&](int i) { return i * kKeys + lane < n ? i * kKeys + lane : i * kKeys; };
        auto page_of = [&](int i) { return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(key_of(i))) * p.page_magic) >> p.page_shift); };
        auto place = [&](int i, int id) {
            const int in = key_of(i) - page_of(i) * p.page_size;
            if (id < 0 || id >= p.num_pages) { id = 0; bad = true; }
            return static_cast<const char *>(p.cache) + (id * p.page_stride + static_cast<int64_t>(in) * p.row_stride) * 2;
        };
        // A step's rows are asked for in thirds: the CU takes 64 bytes a cycle, and all at once (1150
        // cycles) they hold up the waves that ask (12 rows of 64 heads over 280000 keys 272 -> 260 us).
        auto issue = [&](int buf, int third) {
#pragma unroll
            for (int i = third * NC / 3; i < (third + 1) * NC / 3; ++i) {
                const uint32_t at = here(chunk[i]);
                load_to_lds(sh.row[buf][at >> 16] + (at & 0xffffu), lds + buf * (kKeys * DK * 2) + (i * kThreads + wave * 64) * 16);
            }
        };
        lds_barrier();  // the piece before is done with LDS
        if (wave == 0) {
            sh.row[0][lane] = place(s0, table[page_of(s0)]);
            if (count > 1) sh.row[1][lane] = place(s0 + 1, table[page_of(s0 + 1)]);
            if (count > 2) sh.page[0][lane] = table[page_of(s0 + 2)];
        }
        // the queries that the wave multiplies, and what the lane's row sees
        bf16x8 qf[DK / 32];
        const int row = tile * kRows + here(own), t = row / p.H;
        const int limit = min(n, n - p.m + 1 + t);
        {
            const bf16_t *q = static_cast<const bf16_t *>(p.q) + run.b * p.q_sb + t * p.q_st + (row - t * p.H) * p.q_sh;
            const int ch = 8 * here(g);
#pragma unroll
            for (int k = 0; k < DK / 32; ++k) {
                frag8 f;
                f.u = make_uint4(0, 0, 0, 0);
                if (row < rows && 32 * k + ch < d && p.scale != 0.f) f.u = *reinterpret_cast<const uint4 *>(q + 32 * k + ch);
                f.u = make_uint4(f.u.x ^ sign, f.u.y ^ sign, f.u.z ^ sign, f.u.w ^ sign);
                qf[k] = f.v;
            }
        }
        f32x16 acc[NB];
        float top = -INFINITY, top_o = -INFINITY, sum = 0.f;  // the maximum for the lane's row of S^T and of O^T
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = zero16();
        lds_barrier();
#pragma unroll
        for (int k = 0; k < 3; ++k) issue(0, k);
        for (int i = 0, buf = 0; i < count; ++i, buf ^= 1) {
            wait_loads();
            lds_barrier();
            if (i + 1 < count) issue(buf ^ 1, 0);
            if (wave == 0 && i + 3 < count) load_word_to_lds(table + page_of(s0 + i + 3), pages + (buf ^ 1) * (kKeys * 4));
            const char *at = sh.tile[buf];
            const int k0 = (s0 + i) * kKeys + kg * 16 + 4 * g;  // the lane's four keys
            f32x4 s, odd;
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = odd[j] = 0.f;
#pragma unroll
            for (int k = 0; k < DK / 32; ++k) {
                frag8 f;
                f.u = *reinterpret_cast<const uint4 *>(at + (key_at ^ (k & 1 ? 64u : 0u)) + (k >> 1) * 128);
                if (k & 1) odd = mfma16(f.v, qf[k], odd);
                else s = mfma16(f.v, qf[k], s);
            }
            s += odd;
            if (i + 1 < count) issue(buf ^ 1, 1);
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (k0 + j >= limit) s[j] = -INFINITY;
                most = fmaxf(most, s[j]);
            }
            most = quarters_max(most) * c;
            if (g == 0) sh.most[kg][own] = most;
            f32x4 e;
            auto write_p = [&]() {
                const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] = fast_exp2(fmaf(s[j], c, -base));
                f32x4 rest;
#pragma unroll
                for (int j = 0; j < 4; ++j) rest[j] = e[j] - bf16_to_f32(f32_to_bf16(e[j]));
                char *to = sh.p + own * kPRow + (kg * 16 + 4 * g) * 2;
                *reinterpret_cast<uint2 *>(to) = make_uint2(pack2(e[0], e[1]), pack2(e[2], e[3]));
                *reinterpret_cast<uint2 *>(to + kPPart) = make_uint2(pack2(rest[0], rest[1]), pack2(rest[2], rest[3]));
            };
            write_p();
            if (wave == 0 && i + 2 < count) sh.row[buf][lane] = place(s0 + i + 2, sh.page[buf][lane]);
            lds_barrier();
            if (i + 1 < count) issue(buf ^ 1, 2);
            const float all = fmaxf(fmaxf(sh.most[0][c32], sh.most[1][c32]), fmaxf(sh.most[2][c32], sh.most[3][c32]));
            if (__any(all > top_o + kSlack)) {  // the same in every wave
                const float next = fmaxf(top_o, all), keep = next == -INFINITY ? 1.f : fast_exp2(top_o - next);
                top_o = next;
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[b] *= keep;
                const float mine = fmaxf(top, fmaxf(fmaxf(sh.most[0][own], sh.most[1][own]), fmaxf(sh.most[2][own], sh.most[3][own])));
                sum *= mine == -INFINITY ? 1.f : fast_exp2(top - mine);
                top = mine;
                write_p();
                lds_barrier();
            }
            sum += (e[0] + e[1]) + (e[2] + e[3]);
            if (wave * NB * 32 < p.dc) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    frag8 pf, rest;
                    pf.u = *reinterpret_cast<const uint4 *>(sh.p + c32 * kPRow + (16 * k + 8 * h2) * 2);
                    rest.u = *reinterpret_cast<const uint4 *>(sh.p + kPPart + c32 * kPRow + (16 * k + 8 * h2) * 2);
                    // keys 16 k + 8 h2 + 0..3 and + 4..7 in the slots of half h2
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int block = wave * NB + b;
                        const uint32_t turn = block & 1 ? 64u : 0u;
                        const char *from = at + 16 * k * DK * 2 + (block >> 1) * 128;
                        const uint2 lo = read_tr16(from + (value_at ^ turn));
                        const uint2 hi = read_tr16(from + 4 * DK * 2 + (value_at ^ turn ^ 16u));
                        frag8 f;
                        f.u = make_uint4(lo.x, lo.y, hi.x, hi.y);
                        acc[b] = mfma32(f.v, pf.v, acc[b]);
                        acc[b] = mfma32(f.v, rest.v, acc[b]);
                    }
                }
            }
        }
        if (bad && p.status) *p.status = kBadPages;
        // the rows' sums: over the lanes' keys, then over the waves'
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (g == 0) sh.sum[kg][own] = sum;
        lds_barrier();
        const bool whole = count == steps;
        const int in = here(c32), out_row = tile * kRows + in, first_ch = wave * NB * 32 + 4 * here(h2);
        const float all = (sh.sum[0][in] + sh.sum[1][in]) + (sh.sum[2][in] + sh.sum[3][in]);
        const float inv = all == 0.f ? 0.f : 1.f / all;
        if (out_row < rows) {
            const int64_t out = static_cast<int64_t>(run.b) * rows + out_row;
            const int64_t part = (static_cast<int64_t>(tile) * 2 * p.workers + 2 * worker + (first ? 0 : 1)) * kRows + in;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ch = first_ch + 32 * b + 8 * i;
                    if (ch >= p.dc) continue;
                    const f32x4 v = f32x4{acc[b][4 * i], acc[b][4 * i + 1], acc[b][4 * i + 2], acc[b][4 * i + 3]} * inv;
                    if (!whole) *reinterpret_cast<f32x4 *>(p.part_o + part * p.dc + ch) = v;
                    else if constexpr (sizeof(O) == 4) *reinterpret_cast<f32x4 *>(static_cast<O *>(p.o) + out * p.dc + ch) = v;
                    else *reinterpret_cast<uint2 *>(static_cast<O *>(p.o) + out * p.dc + ch) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
                }
            if (wave == 0 && h2 == 0) (whole ? p.lse[out] : p.part_lse[part]) = all == 0.f ? -INFINITY : (top_o + __builtin_amdgcn_logf(all)) * kLn2;
        }
        run.left -= count;
        run.at += count;
        run.before += steps;
        ++run.b;
        first = false;
    }
}

template <typename O, int DK, int DC>
hipError_t run(const LatentDecodeParams &p, const LatentDecodePlan &plan, hipStream_t s) {
    decode_bf16_kernel<O, DK, DC><<<plan.workers * plan.tiles, kThreads, 0, s>>>(p, plan.tiles);
    return hipGetLastError();
}
template <typename O>
hipError_t pick(const LatentDecodeParams &p, const LatentDecodePlan &plan, hipStream_t s) {
    const int d = p.dc + p.dr;
    if (p.dc <= 128 && d <= 192) return run<O, 192, 128>(p, plan, s);
    if (p.dc <= 256 && d <= 320) return run<O, 320, 256>(p, plan, s);
    return run<O, 576, 512>(p, plan, s);
}

}  // namespace

LatentDecodePlan latent_decode_plan(int B, int H, int m, int dc, int dr, int64_t most_rows, int in_dtype) {
    // rows of a tile, keys of a step, workgroups at once
    const bool f32 = in_dtype == 0;
    const int keys = f32 ? kDecodeKeysF32 : kKeys, groups = f32 ? 512 : 256;
    LatentDecodePlan plan{};
    plan.rows = f32 ? kDecodeRowsF32 : kRows;
    plan.tiles = (m * H + plan.rows - 1) / plan.rows;
    // no more workers than there can be steps
    const int64_t most = static_cast<int64_t>(B) * ((most_rows + keys - 1) / keys);
    plan.workers = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, std::max(1, groups / plan.tiles))));
    if (plan.workers > 8) plan.workers = plan.workers / 8 * 8;
    const size_t rows = static_cast<size_t>(plan.tiles) * 2 * plan.workers * plan.rows;
    plan.o_bytes = align_up(rows * dc * sizeof(float));
    plan.lse_bytes = align_up(rows * sizeof(float));
    plan.info_bytes = align_up(static_cast<size_t>(B) * sizeof(int2));
    return plan;
}

hipError_t launch_latent_decode(const LatentDecodeParams &p, const LatentDecodePlan &plan, int in_dtype, int out_dtype, hipStream_t s) {
    const hipError_t e = in_dtype == 0 ? latent_decode_f32(p, plan, out_dtype, s) : out_dtype == 0 ? pick<float>(p, plan, s) : pick<bf16_t>(p, plan, s);
    return e != hipSuccess ? e : launch_latent_join(p, plan, out_dtype, s);
}

}  // namespace kda
