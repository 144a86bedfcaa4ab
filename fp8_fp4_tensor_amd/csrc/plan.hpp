// plan.hpp -- which kernel, tile and split a call of the operators on 8-bit data
// takes: rules on sizes alone, in plain C++ (k_gemm.hip, k_attn.hip; the tests
// compile them without HIP to see that every kernel is reached).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace fq {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------- products
// Which tile, and over how many shares of k. Each tile's time for one step
// (one block of k), in us, alone on its CU and with as many as fit, measured
// on products from 64x2048x7168 to 8192x14336x4096 (bf16 output, and fp32
// with its half-rate products); steps times rounds of workgroups and the
// bytes at 5 TB/s, the longer and a quarter of the other, plus the join's
// launch and traffic, rank the choices. Measured both ways, the tile chosen against the next:
// 2048x4096x4096 128x128 44.6 us, 256x256 55.8; 3000x4096x4096 256x256 57.2,
// 128x128 73.6; 512x4096x14336 128x128 in 4 shares 49.8, whole 105, 64x128 in
// 2 shares 56.1; 16x7168x18432 32x64 in 4 shares 28.2, k_gemm_few 46.6.
struct TileCost {
    int tm, tn, per_cu;
    double alone[2], full[2];  // [bf16, fp32 output]
};
constexpr TileCost kTileCosts[] = {
    {256, 256, 1, {1.75, 3.60}, {1.75, 3.60}},
    {128, 128, 2, {0.94, 1.35}, {1.40, 2.20}},
    {64, 128, 2, {0.67, 0.90}, {1.25, 1.50}},
    {64, 64, 3, {0.60, 0.73}, {1.10, 1.30}},
    {32, 64, 4, {0.42, 0.55}, {1.10, 1.20}},
};
constexpr int kTileKinds = 5;

struct GemmPlan {
    int kind = -1;     // index of kTileCosts, -1: k_gemm_few
    int splits = 1;
    double us = 0.0;   // by the ranking
    int64_t main = 0;  // leading rows that go to 256x256 tiles first, a multiple of 256
};

inline GemmPlan plan_gemm_part(int64_t m, int64_t n, int64_t k, bool bf)
{
    GemmPlan best;
    const int64_t nb = k >> 7;
    // Few rows, at most a workgroup of k_gemm_few a CU and at most 7 blocks a
    // wave: one launch and no LDS (1x4096x4096: 5.4 us, 32x64 tiles 7.7;
    // 1x4096x7168 7.9 and 9.7; beyond it they cross: 1x4096x14336 13.6 and 13.3)
    if ((m <= 16 && n <= 4096 && nb <= 56) || (m <= 16 && n <= 8192 && nb <= 16))
        return best;
    constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
    const int prec = bf ? 0 : 1;
    const double bytes = (double)(m + n) * k + (double)m * n * (bf ? 2 : 4);
    for (int t = 0; t < kTileKinds; ++t) {
        const TileCost& c = kTileCosts[t];
        const int64_t tiles = ceil_div(m, c.tm) * ceil_div(n, c.tn);
        for (int s : kSplits) {
            if (s > 1 && (nb / s < 2 || tiles >= 1024 || (double)s * m * n * 4 > 128e6))
                break;
            const int64_t per_cu = ceil_div(tiles * s, 256);  // workgroups of the busiest CU
            const int64_t rounds = per_cu / c.per_cu, left = per_cu % c.per_cu;
            const double one = c.alone[prec], all = c.full[prec];
            double step = rounds * all;
            if (left)
                step += c.per_cu == 1 ? one : one + (all - one) * (left - 1) / (c.per_cu - 1);
            const double work = ceil_div(nb, s) * step, read = bytes / 5e6;
            double us = work > read ? work + read / 4 : read + work / 4;  // overlapped, but not wholly
            if (s > 1)
                us += 3.0 + (double)s * m * n * 8 / 6e6;
            if (best.kind < 0 || us < best.us) {
                best.kind = t;
                best.splits = s;
                best.us = us;
            }
        }
    }
    return best;
}

// 256x256 tiles that do not come out in whole rounds of the chip leave most of
// it idle in the last one: the rows beyond the whole rounds are then a product
// of their own, with the tile and shares that suit it (14336x4096x8192, fp32:
// 3.5 rounds as 3 and 128x128 tiles).
inline GemmPlan plan_gemm(int64_t m, int64_t n, int64_t k, bool bf)
{
    GemmPlan best = plan_gemm_part(m, n, k, bf);
    const int64_t across = ceil_div(n, 256), whole = ceil_div(m, 256) * across / 256;
    if (best.kind != 0 || best.splits > 1 || whole < 1)
        return best;
    const int64_t main = whole * 256 / across * 256;  // rows of `whole` rounds
    if (main == 0 || main >= m)
        return best;
    GemmPlan rest = plan_gemm_part(m - main, n, k, bf);
    rest.us += plan_gemm_part(main, n, k, bf).us + 2.0;
    if (rest.kind < 0 || rest.us >= best.us)
        return best;
    rest.main = main;
    return rest;
}

// ---------------------------------------------------------------- attention
constexpr int kAttnStep = 64;     // keys a step of a wave takes
constexpr int kAttnRows = 16;     // query rows of a workgroup of the kernel for few rows
constexpr int kAttnSplits = 512;  // the most shares of a sequence

// Query rows of a workgroup of the kernel for many rows, eight waves: 32 a wave,
// 16 with 256 dims.
constexpr int attn_tile_rows(int dim) { return dim == 256 ? 128 : 256; }

struct AttnPlan {
    int rows = kAttnRows;  // query rows of a workgroup: kAttnRows, or attn_tile_rows
    int tiles = 0;         // row tiles of the longest run of queries
    int waves = 4;         // of a workgroup for few rows
    int chunk = 0;         // keys a share
    int splits = 1;        // shares of the longest sequence
};

inline AttnPlan plan_attention(int64_t batch, int64_t heads, int64_t q_heads, int dim, int64_t max_q, int64_t max_len,
                               int64_t window)
{
    AttnPlan p;
    const int64_t group = q_heads / heads;
    // The kernel for many rows, where its workgroups fill the chip and their
    // rows: a step of 64 keys costs it the same up to 256 workgroups, and the
    // kernel for few rows in proportion to its tiles of 16 rows. They are even at
    // the tiles below, measured with 32 heads over 8, many against few in us: 128
    // dims, 8 sequences of 128 rows and up to 2000 keys (2048 tiles) 71 and 88; 6
    // of them (1536) 70 and 67; 2 of 320 rows and 8192 keys (1280) 252 and 224;
    // 2 of 400 rows and 2000 keys (1600) 69 and 81; 64 dims, 8 of 128 rows (2048)
    // 57 and 42; 256 dims, 4 of 128 rows (1024) 86 and 123.
    const int64_t even = dim == 64 ? 2800 : dim == 128 ? 1600 : 725;
    const int64_t wide = attn_tile_rows(dim);
    const int64_t few_tiles = batch * heads * ceil_div(max_q * group, kAttnRows);
    const int64_t many_tiles = batch * heads * ceil_div(max_q * group, wide);
    if (ceil_div(many_tiles, 256) * even < few_tiles) {
        p.rows = (int)wide;
        p.tiles = (int)ceil_div(max_q * group, wide);
        p.chunk = (int)max_len;
        p.splits = 1;
        return p;
    }
    p.tiles = (int)ceil_div(max_q * group, kAttnRows);
    const int64_t tiles = batch * heads * p.tiles;
    int64_t span = max_len;
    if (window > 0 && span > window + max_q + kAttnStep)
        span = window + max_q + kAttnStep;
    // One workgroup per tile if the tiles alone fill the chip, else about two
    // workgroups a CU, each with at least a step for each of its four waves
    // (4 sequences of up to 131072: 16 splits 164 us, 32 177, 64 169, 128 171;
    // 64 of up to 8192: one 119 us, two 131, eight 120). A short run of keys
    // on few tiles stays whole, on eight waves: no second launch.
    int64_t splits = tiles >= 512 ? 1 : ceil_div(512, tiles > 0 ? tiles : 1);
    if (splits > 1 && span <= 1024 && dim <= 128) {
        p.waves = 8;
        splits = 1;
    }
    if (span < 1)
        span = 1;
    const int64_t chunk = ceil_div(ceil_div(span, splits), 4 * kAttnStep) * (4 * kAttnStep);
    p.chunk = (int)chunk;
    p.splits = (int)ceil_div(span, chunk);
    return p;
}

}  // namespace fq
