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

// ---------------------------------------------------------------- products of MX planes
constexpr int kChipCus = 256;

// Tiles, and the time of one step (128 bytes of a row; 128 elements with one
// 4-bit side) in us, alone on a CU and with as many as fit: both sides 8-bit,
// both 4-bit, one of each, and widened (fp32 results with an 8-bit side).
// From outputs of one round of the chip and depths of 2048 and 6144.
struct MxTileCost {
    int tm, tn, per_cu;
    double alone[4], full[4];
};
constexpr MxTileCost kMxTiles[] = {
    {256, 256, 1, {1.60, 1.90, 1.56, 2.75}, {1.60, 1.90, 1.56, 2.75}},
    {128, 256, 1, {1.15, 1.41, 1.03, 1.60}, {1.15, 1.41, 1.03, 1.60}},
    {64, 128, 2, {0.50, 0.63, 0.47, 0.73}, {1.03, 1.18, 0.97, 1.22}},
    {64, 64, 3, {0.36, 0.43, 0.34, 0.56}, {0.98, 1.08, 0.90, 1.16}},
};
constexpr int kMxTileKinds = 4;

struct MxPlan {
    int kind = -1;     // index of kMxTiles, -1: k_gemm_mx_few
    int splits = 1;
    double us = 0.0;   // by the ranking
    int64_t main = 0;  // leading rows that go to 256x256 tiles first, a multiple of 256
    bool arranged = false;  // scales are laid out for the tiles first
};

// The ranking is plan_gemm_part's: steps times rounds of workgroups and the
// bytes at 6.3 TB/s, the longer and a quarter of the other, plus the join of
// shares. Measured both ways, what is chosen first (us; 8-bit both sides and
// bf16 results where nothing is said):
//   1x4096x4096        few rows 7.5, 64x64 in 8 shares 7.1; 4-bit B 4.3 and 6.8
//   16x8192x8192       64x128 in 8 shares 16.0, 64x64 in 4 15.0, few rows 23.8
//   16x18432x7168      64x128 in 3 shares 31.4, in 8 31.2
//   48x18432x7168      64x128 in 3 shares 37.4, 128x256 in 3 38.9; 4-bit 21.3, whole 19.7
//   256x4096x4096      64x64 14.7, 64x128 18.3
//   1003x7168x2048     128x256 21.7, 256x256 27.5, 64x128 28.0
//   512x4096x14336     128x256 in 4 shares 48.2, 256x256 in 6 51.1, 64x128 57.1
//   4096x4096x4096     256x256 59, 128x256 73; 4-bit 42.5 and 50.7; fp32 104 and 119
//   14336x4096x8192    fp32: three rounds of 256x256 and the rest on 128x256 697, all on 256x256 703, on 128x256 771
// Over 130 shapes the choice takes 4.0% longer than the best (geometric mean), at worst 1.35 times as long (20x8848x3840,
// 4-bit, fp32 results: 64x128 in 6 shares 12.3, 64x64 9.1).
inline MxPlan plan_gemm_mx_part(int64_t m, int64_t n, int64_t k, bool a4, bool b4, bool bf)
{
    MxPlan best;
    const int cost = a4 && b4 ? 1 : !bf ? 3 : a4 || b4 ? 2 : 0;
    const int64_t steps = ceil_div(k, a4 && b4 ? 256 : 128);
    constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
    const double bytes = (double)m * (a4 ? k / 2 : k) + (double)n * (b4 ? k / 2 : k) + (double)(m + n) * k / 32 +
                         (double)m * n * (bf ? 2 : 4);
    // few rows, and a workgroup of k_gemm_mx_few a CU or little of B: one launch and no LDS (12x9104x1152, 4-bit: 3.6
    // us, 64x64 4.7). The border is not exact: beyond it 1x14336x4096 with 4-bit B takes 14.1 (64x128 in 16 shares) and
    // few rows 11.3, 7x7616x7424 in 4 bits 11.6 and 9.7; within it 2x1112x16256 with 4-bit B 10.2, 64x64 in 12 shares 8.8.
    if (m <= 16 && ((n <= 4096 && k <= 16384) || (double)n * (b4 ? k / 2 : k) <= 9e6))
        return best;
    for (int t = 0; t < kMxTileKinds; ++t) {
        const MxTileCost& c = kMxTiles[t];
        const int64_t tiles = ceil_div(m, c.tm) * ceil_div(n, c.tn);
        // one row of tiles takes B from memory and not from L2
        const double one = c.alone[cost] * (c.per_cu > 1 && m <= c.tm ? 1.5 : 1.0), all = c.full[cost];
        for (int s : kSplits) {
            if (s > 1 && (steps / s < 2 || tiles >= 1024 || (double)s * m * n * 4 > 128e6))
                break;
            const int64_t per_cu = ceil_div(tiles * s, kChipCus);  // workgroups of the busiest CU
            const int64_t rounds = per_cu / c.per_cu, left = per_cu % c.per_cu;
            double step = rounds * all;
            if (left)
                step += c.per_cu == 1 || one > all ? one : one + (all - one) * (left - 1) / (c.per_cu - 1);
            const double work = ceil_div(steps, s) * step, read = bytes / 6.3e6;
            double us = work > read ? work + read / 4 : read + work / 4;  // overlapped, but not wholly
            if (s > 1)
                us += 4.5 + (double)s * m * n * 8 / 6e6;
            if (best.kind < 0 || us < best.us) {
                best.kind = t;
                best.splits = s;
                best.us = us;
            }
        }
    }
    return best;
}

inline MxPlan plan_gemm_mx(int64_t m, int64_t n, int64_t k, bool a4, bool b4, bool bf)
{
    MxPlan best = plan_gemm_mx_part(m, n, k, a4, b4, bf);
    // rows beyond whole rounds of 256x256 tiles, as in plan_gemm
    const int64_t across = ceil_div(n, 256), whole = ceil_div(m, 256) * across / kChipCus;
    if (best.kind == 0 && best.splits == 1 && whole >= 1) {
        const int64_t main = whole * kChipCus / across * 256;
        if (main > 0 && main < m) {
            MxPlan rest = plan_gemm_mx_part(m - main, n, k, a4, b4, bf);
            rest.us += plan_gemm_mx_part(main, n, k, a4, b4, bf).us + 2.0;
            if (rest.kind >= 0 && rest.us < best.us) {  // not k_gemm_mx_few: it takes no laid out scales
                best = rest;
                best.main = main;
            }
        }
    }
    // Scales that a 256x256 tile takes from a plane are a line of memory for
    // each row, word and step, half as many again as the operands (with 4-bit
    // sides as many again). Laid out by rows first they are 1 KB in a piece,
    // which saves about 0.18 us a step (0.3, and 0.115 with one 4-bit side) and
    // costs a launch of 5 us or more; with widened operands it saves nothing.
    //   8192x14336x4096  8-bit 382 us, 452 without; 4-bit 261, 294; one of each 368, 387
    //   4096x14336x4096  8-bit 211, 252; 4-bit 133, 148
    //   4096x4096x7168   8-bit 95.0, 96.3;  4096x4096x5120  73.7, 73.5;  4096x4096x4096  64.0, 61.3
    //   8192x4096x4096   4-bit 79.6, 80.9;  4096x4096x4096  45.0, 42.6
    //   4096x4096x14336  one of each 164, 172;  8192x8192x2048  121.9, 120.7
    //   18432x7168x2048  4-bit 169, 161 without: eight steps, and results that take as long to write
    // A plane whose rows of scales are no whole words needs it whatever the size.
    const int cost = a4 && b4 ? 1 : !bf ? 3 : a4 || b4 ? 2 : 0;
    constexpr double kSaves[] = {0.18, 0.30, 0.115, 0.0};
    const int64_t steps = ceil_div(k, a4 && b4 ? 256 : 128);
    const int64_t rounds = ceil_div(ceil_div(best.main ? best.main : m, 256) * across, kChipCus);
    const bool large = best.main || (best.kind == 0 && best.splits == 1);
    best.arranged = best.kind >= 0 && (k % 128 != 0 || (large && steps >= 12 && kSaves[cost] * rounds * steps > 7.5));
    return best;
}

// ---------------------------------------------------------------- planes
// Bytes that a store of a tile's MX scales takes at a time: a row's (column's)
// `codes` of them start at code `first` of a row of `per`, and each store has to
// lie on its own size. The second half of a gated activation's gradient starts
// at any code.
constexpr int scale_store_bytes(int64_t per, int64_t first, int codes)
{
    return codes != 4 ? 1 : ((per | first) & 3) == 0 ? 4 : ((per | first) & 1) == 0 ? 2 : 1;
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
