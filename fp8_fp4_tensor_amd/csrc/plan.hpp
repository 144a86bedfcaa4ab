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
// on products from 64x2048x7168 to 8192x14336x4096: bf16 output with 128x128
// scales, and fp32 output with 1x128 scales, the weight gradient's, with its
// half-rate products (256x256 tiles, by 4096x4096 outputs of depths 2048 and
// 14336: 1.79 and 3.67; the other two ways around 2.29 and 3.23). Steps times
// rounds of workgroups and the bytes at 5 TB/s, the longer and a quarter of
// the other, plus the join's launch and traffic, rank the choices. Measured
// both ways, what is chosen first (us):
//   2048x4096x4096    128x128 48.2, 256x256 56.4
//   3000x4096x4096    256x256 57.9, 128x128 78.0
//   1003x7168x2048    128x128 26.9, 256x256 32.1, 64x128 34.6
//   512x4096x14336    256x256 in 8 shares 57.0, 128x128 in 4 60.8, whole 131
//   48x18432x7168     64x128 in 3 shares 36.9, whole 40.8, in 2 45.4
//   16x7168x18432     32x64 in 6 shares 31.1, k_gemm_few 46.1
// The ranking is not exact: 4 shares of the last would take 28.7.
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
    // wave: one launch and no LDS (1x4096x4096: 6.7 us, 32x64 tiles 8.9;
    // 1x4096x7168 7.9 and 9.8; beyond it little is between them: 1x4096x14336
    // 13.6, and 14.3 to 15.1 by shares)
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
// 3.5 rounds as 3 and 256x256 tiles in two shares 883 us, all on whole 256x256
// tiles 914, on 128x128 992).
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
    // kernel for few rows in proportion to its tiles of 16 rows. Many against few
    // in us, sequences of 256 or 512 rows (tokens times group) and up to 2000 keys:
    //   64 dims    2048 tiles 56.4 and 49.9, 2560 56.3 and 58.4, 2816 56.5 and 62.6;
    //              with a cap 2560 72.7 and 70.8, 2816 72.5 and 74.9
    //   128 dims   1280 tiles 69.3 and 64.2, 1536 69.6 and 73.0, 1792 69.7 and 83.0;
    //              with a cap 1536 85.7 and 78.0, 1792 85.9 and 89.8
    //   256 dims   512 tiles 86.5 and 76.5, 640 86.9 and 102.7, 768 86.6 and 110;
    //              with a cap 512 95.5 and 81.8, 768 95.6 and 117
    // (groups of 1 and of 8 within 2% of groups of 4). The borders stand at or above
    // what is even, for the kernel for few rows rounds its probabilities less.
    const int64_t border = dim == 64 ? 2800 : dim == 128 ? 1600 : 725;
    const int64_t wide = attn_tile_rows(dim);
    const int64_t few_tiles = batch * heads * ceil_div(max_q * group, kAttnRows);
    const int64_t many_tiles = batch * heads * ceil_div(max_q * group, wide);
    if (ceil_div(many_tiles, 256) * border < few_tiles) {
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
