// Latent attention's absorbed form on the bf16 matrix cores.
//
// A workgroup of eight waves takes ROWS rows (token, head) of a sequence, 32 or
// 64, and a run of the cache, 64 rows (keys) a step, which come from memory to LDS
// directly, one step ahead: 74 KB in flight on every CU.  A step's rows are read
// twice, by rows as keys and by columns as values.
//   S^T = K Q^T    wave w: keys 16 (w % 4), ROWS / 2 rows (w / 4), all channels
//                  (16 x 16 x 32 products; Q stays in registers)
//   softmax        the waves' maxima meet in LDS; P, bf16, goes there too
//   O^T += C^T P^T wave w: an eighth of the latent channels, all rows
//                  (32 x 32 x 16 products)
// With 32 rows (one token of up to 32 heads) a step's arithmetic takes about a
// quarter of the time of its bytes; with many more rows the products are the bound
// and 64 rows halve the reads of LDS for each.
#include "kda_latent_bf16.hpp"
#include "kda_latent_decode.hpp"

namespace kda {

namespace {

constexpr int kKeys = 64, kThreads = 512;
constexpr float kSlack = 8.f;       // see the forward: how far P may pass 1 (log2)
constexpr int kPRow = kKeys * 2 + 16;  // bytes of a row of P: 16 more than its keys

// chunk c of row r of the tile (read by rows and by columns)
__device__ __forceinline__ constexpr int swizzle(int r, int c) { return (c & ~7) | ((c ^ r ^ (r >> 3 & 1)) & 7); }

template <int DK, int DC, int ROWS> struct Shared {
    char tile[2][kKeys * DK * 2];
    char p[ROWS * kPRow];
    float most[4][ROWS];     // each 16 keys' maximum
    float sum[4][ROWS];
    const char *row[2][kKeys];
    int64_t steps[kThreads / 64];
};

template <typename O, int DK, int DC, int ROWS>
__global__ void __launch_bounds__(kThreads, 1) decode_bf16_kernel(LatentDecodeParams p, int tiles) {
    constexpr int NC = kKeys * DK / 8 / kThreads;   // chunks a thread
    constexpr int NB = DC / 8 / 32 ? DC / 8 / 32 : 1;  // 32-channel blocks a wave
    constexpr int NR = ROWS / 32;                   // 16-row blocks of the scores, 32-row blocks of the result
    __shared__ __attribute__((aligned(16))) Shared<DK, DC, ROWS> sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c16 = lane & 15, h2 = lane >> 5, c32 = lane & 31;
    const int kg = wave & 3, rg = wave >> 2;        // the wave's keys and rows of S^T
    int tile, worker;
    if (p.workers % 8 == 0) {  // the row tiles of one worker on one XCD: they read the same rows
        const int x = blockIdx.x >> 3;
        tile = x % tiles;
        worker = (x / tiles) * 8 + (blockIdx.x & 7);
    } else {
        tile = blockIdx.x % tiles;
        worker = blockIdx.x / tiles;
    }
    DecodeRun run = decode_run<kThreads, kKeys>(p, worker, sh.steps);
    const int d = p.dc + p.dr, rows = p.m * p.H;
    const float c = p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e;
    const uint32_t sign = p.scale < 0.f ? 0x80008000u : 0u;

    uint32_t chunk[NC];  // (row of the tile, byte of its channels) of the thread's chunks
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int at = i * kThreads + tid, r = at / (DK / 8), ch = swizzle(r, at % (DK / 8)) * 8;
        chunk[i] = static_cast<uint32_t>(r) << 16 | static_cast<uint32_t>(ch < d ? ch * 2 : 0);  // channels behind the last meet zeros of q
    }
    const uint32_t lds = lds_address(sh.tile[0]);
    // the lane's bytes in a tile: its key's row, chunk g (the even steps; bit 2 of the chunk is the step's)
    const uint32_t key_at = static_cast<uint32_t>(kg * 16 + c16) * (DK * 2) + swizzle(c16, g) * 16;
    // .. and its four channels of row c16 / 4 of a half's eight (rows 4 further: bit 2 of the chunk turns)
    const uint32_t value_at = static_cast<uint32_t>(8 * h2 + (c16 >> 2)) * (DK * 2) + swizzle(8 * h2 + (c16 >> 2), 2 * (g & 1) + ((c16 & 3) >> 1)) * 16 + 8 * (c16 & 1);

    bool first = true;
    while (run.left > 0) {
        const int n = decode_rows(p, run.b);
        const int64_t steps = (n + kKeys - 1) / kKeys;
        if (steps == 0) { ++run.b; continue; }
        const int s0 = first ? static_cast<int>(run.at - run.before) : 0;
        const int count = static_cast<int>(min(run.left, steps - s0));
        if (s0 == 0 && tile == 0 && tid == 0) p.info[run.b] = decode_info(first, run.per, run.before, steps, worker);

        // the place of row `lane` of step i (a row behind the last stands for the step's first: its weight is 0)
        const int32_t *table = p.page_table + run.b * p.table_stride;
        bool bad = p.lengths[run.b] != n;
        auto place = [&](int i) {
            const int k0 = i * kKeys, k = k0 + lane < n ? k0 + lane : k0;
            const int page = k / p.page_size;
            int id = table[page];
            if (id < 0 || id >= p.num_pages) { id = 0; bad = true; }
            return static_cast<const char *>(p.cache) + (id * p.page_stride + static_cast<int64_t>(k - page * p.page_size) * p.row_stride) * 2;
        };
        auto issue = [&](int buf) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                load_to_lds(sh.row[buf][chunk[i] >> 16] + (chunk[i] & 0xffffu), lds + buf * (kKeys * DK * 2) + (i * kThreads + wave * 64) * 16);
        };
        lds_barrier();  // the piece before is done with LDS
        if (wave == 0) sh.row[0][lane] = place(s0);
        if (wave == 0 && count > 1) sh.row[1][lane] = place(s0 + 1);
        // the queries that the wave multiplies, and what its lanes' rows see
        bf16x8 qf[NR][DK / 32];
        int limit[NR];
        const bf16_t *q = static_cast<const bf16_t *>(p.q) + run.b * p.q_sb;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = tile * ROWS + rg * (ROWS / 2) + 16 * r + c16, t = row / p.H;
            limit[r] = min(n, n - p.m + 1 + t);
            const bf16_t *qr = q + t * p.q_st + (row - t * p.H) * p.q_sh;
#pragma unroll
            for (int k = 0; k < DK / 32; ++k) {
                frag8 f;
                f.u = make_uint4(0, 0, 0, 0);
                if (row < rows && 32 * k + 8 * g < d && p.scale != 0.f) f.u = *reinterpret_cast<const uint4 *>(qr + 32 * k + 8 * g);
                f.u = make_uint4(f.u.x ^ sign, f.u.y ^ sign, f.u.z ^ sign, f.u.w ^ sign);
                qf[r][k] = f.v;
            }
        }
        f32x16 acc[NB][NR];
        float top[NR], top_o[NR], sum[NR];  // of the score rows' lanes, and of the result's
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            top[r] = top_o[r] = -INFINITY;
            sum[r] = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[b][r] = zero16();
        }
        lds_barrier();
        issue(0);
        const char *ahead = nullptr;
        for (int i = 0, buf = 0; i < count; ++i, buf ^= 1) {
            wait_loads();
            lds_barrier();
            if (i + 1 < count) issue(buf ^ 1);
            if (wave == 0 && i + 2 < count) ahead = place(s0 + i + 2);
            const char *at = sh.tile[buf];
            const int k0 = (s0 + i) * kKeys;
            f32x4 s[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) s[r] = f32x4{0.f, 0.f, 0.f, 0.f};
            {
#pragma unroll
                for (int k = 0; k < DK / 32; ++k) {
                    frag8 f;
                    f.u = *reinterpret_cast<const uint4 *>(at + (key_at ^ (k & 1 ? 64u : 0u)) + (k >> 1) * 128);
#pragma unroll
                    for (int r = 0; r < NR; ++r) s[r] = mfma16(f.v, qf[r][k], s[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float most = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k0 + kg * 16 + 4 * g + j >= limit[r]) s[r][j] = -INFINITY;
                    most = fmaxf(most, s[r][j]);
                }
                most = fmaxf(most, __shfl_xor(most, 16));
                most = fmaxf(most, __shfl_xor(most, 32));
                if (g == 0) sh.most[kg][rg * (ROWS / 2) + 16 * r + c16] = most * c;
            }
            lds_barrier();
            if (wave == 0 && i + 2 < count) sh.row[buf][lane] = ahead;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int in = rg * (ROWS / 2) + 16 * r + c16;
                const float most = fmaxf(fmaxf(sh.most[0][in], sh.most[1][in]), fmaxf(sh.most[2][in], sh.most[3][in]));
                if (most > top[r] + kSlack) {
                    sum[r] *= fast_exp2(top[r] - most);
                    top[r] = most;
                }
                const float base = top[r] == -INFINITY ? 0.f : top[r];
                uint32_t w[2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[r][j] = fast_exp2(fmaf(s[r][j], c, -base));
                    sum[r] += s[r][j];
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) w[j] = static_cast<uint32_t>(f32_to_bf16(s[r][2 * j])) | static_cast<uint32_t>(f32_to_bf16(s[r][2 * j + 1])) << 16;
                *reinterpret_cast<uint2 *>(sh.p + in * kPRow + (kg * 16 + 4 * g) * 2) = make_uint2(w[0], w[1]);
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int in = 32 * r + c32;
                const float most = fmaxf(fmaxf(sh.most[0][in], sh.most[1][in]), fmaxf(sh.most[2][in], sh.most[3][in]));
                const bool moves = most > top_o[r] + kSlack;
                if (__any(moves)) {
                    const float keep = moves ? fast_exp2(top_o[r] - most) : 1.f;
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[b][r] *= keep;
                }
                if (moves) top_o[r] = most;
            }
            lds_barrier();
            if (wave * NB * 32 < p.dc) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bf16x8 pf[NR];
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        frag8 f;
                        f.u = *reinterpret_cast<const uint4 *>(sh.p + (32 * r + c32) * kPRow + (16 * k + 8 * h2) * 2);
                        pf[r] = f.v;
                    }
                    // keys 16 k + 8 h2 + 0..3 and + 4..7 in the slots of half h2
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int block = wave * NB + b;
                        const uint32_t turn = block & 1 ? 64u : 0u;
                        const char *from = at + 16 * k * DK * 2 + (block >> 1) * 128;
                        const uint2 lo = read_tr16(from + (value_at ^ turn));
                        const uint2 hi = read_tr16(from + 4 * DK * 2 + (value_at ^ turn ^ 64u));
                        frag8 f;
                        f.u = make_uint4(lo.x, lo.y, hi.x, hi.y);
#pragma unroll
                        for (int r = 0; r < NR; ++r) acc[b][r] = mfma32(f.v, pf[r], acc[b][r]);
                    }
                }
            }
        }
        if (bad && p.status) *p.status = kBadPages;
        // the rows' sums: over the lanes' keys, then over the waves'
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            sum[r] += __shfl_xor(sum[r], 16);
            sum[r] += __shfl_xor(sum[r], 32);
            if (g == 0) sh.sum[kg][rg * (ROWS / 2) + 16 * r + c16] = sum[r];
        }
        lds_barrier();
        const bool whole = count == steps;
        const int64_t slot = static_cast<int64_t>(tile) * 2 * p.workers + 2 * worker + (first ? 0 : 1);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int in = 32 * r + c32, row = tile * ROWS + in;
            const float all = (sh.sum[0][in] + sh.sum[1][in]) + (sh.sum[2][in] + sh.sum[3][in]);
            const float inv = all == 0.f ? 0.f : 1.f / all;
            if (row >= rows) continue;
            const int64_t out = static_cast<int64_t>(run.b) * rows + row, part = slot * ROWS + in;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ch = (wave * NB + b) * 32 + 8 * i + 4 * h2;
                    if (ch >= p.dc) continue;
                    const f32x4 v = f32x4{acc[b][r][4 * i], acc[b][r][4 * i + 1], acc[b][r][4 * i + 2], acc[b][r][4 * i + 3]} * inv;
                    if (!whole) {
                        *reinterpret_cast<f32x4 *>(p.part_o + part * p.dc + ch) = v;
                    } else if constexpr (sizeof(O) == 4) {
                        *reinterpret_cast<f32x4 *>(static_cast<O *>(p.o) + out * p.dc + ch) = v;
                    } else {
                        uint32_t w[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) w[j] = static_cast<uint32_t>(f32_to_bf16(v[2 * j])) | static_cast<uint32_t>(f32_to_bf16(v[2 * j + 1])) << 16;
                        *reinterpret_cast<uint2 *>(static_cast<O *>(p.o) + out * p.dc + ch) = make_uint2(w[0], w[1]);
                    }
                }
            if (wave == 0 && h2 == 0) (whole ? p.lse[out] : p.part_lse[part]) = all == 0.f ? -INFINITY : (top_o[r] + __builtin_amdgcn_logf(all)) * kLn2;
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
    const int grid = plan.workers * plan.tiles;
    if (plan.rows == 32) decode_bf16_kernel<O, DK, DC, 32><<<grid, kThreads, 0, s>>>(p, plan.tiles);
    else decode_bf16_kernel<O, DK, DC, 64><<<grid, kThreads, 0, s>>>(p, plan.tiles);
    return hipGetLastError();
}
template <typename O>
hipError_t pick(const LatentDecodeParams &p, const LatentDecodePlan &plan, hipStream_t s) {
    const int d = p.dc + p.dr;
    if (p.dc <= 128 && d <= 192) return run<O, 192, 128>(p, plan, s);
    if (p.dc <= 256 && d <= 320) return run<O, 320, 256>(p, plan, s);
    return run<O, 576, 512>(p, plan, s);
}

// rows of a tile, rows a step, workgroups at once
struct Shape { int rows, keys, groups; };
Shape shape(int rows, int in_dtype) {
    if (in_dtype == 0) return {kDecodeRowsF32, kDecodeKeysF32, 512};
    return {rows <= 32 ? 32 : 64, kKeys, 256};
}

}  // namespace

LatentDecodePlan latent_decode_plan(int B, int H, int m, int dc, int dr, int64_t most_rows, int in_dtype) {
    const Shape sh = shape(m * H, in_dtype);
    LatentDecodePlan plan{};
    plan.rows = sh.rows;
    plan.tiles = (m * H + plan.rows - 1) / plan.rows;
    // as many as run at once, and no more than there can be steps
    const int64_t most = static_cast<int64_t>(B) * ((most_rows + sh.keys - 1) / sh.keys);
    plan.workers = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, std::max(1, sh.groups / plan.tiles))));
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
