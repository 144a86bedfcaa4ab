// k_gemm_mx.hip -- the matrix product of MX planes on gfx950.
//
//   C[i, j] = sum_b 2^(ea[i, b] - 127) 2^(eb[j, b] - 127) sum_{t < 32} A[i, 32 b + t] B[j, 32 b + t]
//
// A: [m, k] and B: [n, k] codes, E4M3, E5M2 or E2M1 on either side, with one
// E8M0 code for 32 elements of a row. Both run along k, and the matrix
// instruction applies the scales, so a product is nothing but operands in and
// sums out.
//
// A few rows take a kernel without LDS tiles or a second launch (1x4096x4096,
// 8-bit times 4-bit: 4.2 us, two latencies of memory and a launch), others tiles
// (gemm_mx_tile.hpp).
//
// Operand order: B's rows are the instruction's rows and A's rows its columns,
// so a lane holds one row i of C and four consecutive columns j.
#include "gemm_mx.hpp"
#include "mx_operand.hpp"
#include "plan.hpp"

namespace fq {
namespace {

// One workgroup computes 16x16 outputs; its waves take pairs of 128 elements
// of k in turn and their sums meet in LDS, in wave order.
constexpr int kFewWaves = 8;

// The operand of a lane: 128 elements from element k0 of the row at p, zeros past k.
template <int F, bool WIDE>
__device__ __forceinline__ i32x8 load128(const uint8_t* p, int64_t k0, int64_t k, int g, bool stream)
{
    const u32x4 zero = {0u, 0u, 0u, 0u};
    auto ld = [&](int64_t at) { return stream ? ld16_stream(p + at) : ld16(p + at); };
    if constexpr (F == kE2M1) {
        const int64_t at = k0 + 32 * g;
        return join(at < k ? ld(at >> 1) : zero, zero);
    } else {
        // widened: whole blocks, as a 4-bit side has them
        const int64_t lo = k0 + (WIDE ? 32 * g : 16 * g), hi = WIDE ? lo + 16 : lo + 64;
        return join(lo < k ? ld(lo) : zero, hi < k ? ld(hi) : zero);
    }
}

template <int FA, int FB, bool WIDE>
__global__ __launch_bounds__(kFewWaves * 64) void k_gemm_mx_few(GemmMxArgs a)
{
    __shared__ f32x4 part[kFewWaves][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16;
    const int64_t nb = a.k >> 5;
    // rows and columns past the last repeat it and are not stored
    const int64_t i = min(m0 + row, a.m - 1), j = min(n0 + row, a.n - 1);
    const uint8_t* pa = a.a + mx_bytes<FA>(i * a.k);
    const uint8_t* pb = a.b + mx_bytes<FB>(j * a.k);
    const uint8_t* psa = a.sa + i * nb;
    const uint8_t* psb = a.sb + j * nb;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t k0 = 256 * w; k0 < a.k; k0 += 256 * kFewWaves) {
        i32x8 fa[2], fb[2];
        uint32_t sa[2], sb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t b = min((k0 + 128 * h) / 32 + g, nb - 1);
            fb[h] = load128<FB, WIDE>(pb, k0 + 128 * h, a.k, g, true);
            fa[h] = load128<FA, WIDE>(pa, k0 + 128 * h, a.k, g, false);
            sb[h] = psb[b];
            sa[h] = psa[b];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (WIDE) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<FB>(fb[h], e, e8m0_value(sb[h])),
                                                                  widen8<FA>(fa[h], e, e8m0_value(sa[h])), acc, 0, 0, 0);
            } else {
                acc = mfma_mx<FB, FA>(fb[h], sb[h], fa[h], sa[h], acc);
            }
        }
    }
    if constexpr (WIDE) {
        // as in the tiles: this wave's sums that are not finite, where a row's scales can be the cause
        float zero = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            zero = __builtin_fmaf(acc[e], 0.0f, zero);
        if (__ballot(zero != 0.0f) != 0) {
            const int far_a = past_top<FA, 16>(psa, 0, nb, g), far_b = past_top<FB, 16>(psb, 0, nb, g);
            if (__ballot((far_a | far_b) != 0) != 0) {
                f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int64_t b0 = 8 * w; b0 < nb; b0 += 8 * kFewWaves)
                    for (int64_t b = b0; b < min(b0 + 8, nb); ++b)
                        add_block<FA, FB, 16>(pa, psa, pb, psb, b, g, sum);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((far_a | __shfl(far_b, row_of_sum<16>(e, g))) && no_number(acc[e]))
                        acc[e] = sum[e];
            }
        }
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w > 0 || m0 + row >= a.m)
        return;
#pragma unroll
    for (int x = 1; x < kFewWaves; ++x)
        acc += part[x][lane];
    if (a.bf)
        store4<true>(a.c, m0 + row, n0 + g * 4, a.n, acc, false);
    else
        store4<false>(a.c, m0 + row, n0 + g * 4, a.n, acc, a.acc);
}

template <int FA, int FB>
hipError_t few(const GemmMxArgs& a, hipStream_t st)
{
    const dim3 grid((unsigned)cdiv(a.n, 16), (unsigned)cdiv(a.m, 16));
    constexpr int th = kFewWaves * 64;
    if (kWidened<FA, FB, true> && !a.bf)
        k_gemm_mx_few<FA, FB, kWidened<FA, FB, true>><<<grid, th, 0, st>>>(a);
    else
        k_gemm_mx_few<FA, FB, false><<<grid, th, 0, st>>>(a);
    return hipGetLastError();
}

// Scales [rows, nb] of both operands -> words as MxTileArgs has them, zeros past
// nb and past the last row of a group of 64: a wave takes 64 words of a group.
struct ScalesArgs {
    const uint8_t* from[2];
    uint32_t* to[2];
    int64_t rows[2], groups_a;
    int nb, words;
};

__global__ __launch_bounds__(kWG) void k_gemm_mx_scales(ScalesArgs a)
{
    __shared__ uint32_t tile[64][65];
    const int64_t group = blockIdx.x;
    const int which = group < a.groups_a ? 0 : 1;
    const int64_t g = which ? group - a.groups_a : group;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int first = blockIdx.y * 64, word = first + lane;
    // All loads first: each in a branch of its own would wait for the one before (8192x14336x4096, 4-bit: 12 us, 5.2 so;
    // 14336x4096x8160, whose rows of 255 scales start anywhere: 16 us). A row's last word reaches back into the one
    // before and is shifted; rows past the last repeat it and count as zeros.
    uint32_t v[16];
    auto row_of = [&](int i) { return a.from[which] + min(g * 64 + w * 16 + i, a.rows[which] - 1) * a.nb; };
    if (a.nb >= 4) {
        const int from = min(4 * word, a.nb - 4);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            __builtin_memcpy(&v[i], row_of(i) + from, 4);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] >>= min(8 * (4 * word - from), 31);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v[i] = 0;
#pragma unroll
            for (int e = 0; e < 3; ++e)
                v[i] |= e < a.nb ? (uint32_t)row_of(i)[e] << 8 * e : 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        tile[w * 16 + i][lane] = g * 64 + w * 16 + i < a.rows[which] && word < a.words ? v[i] : 0u;
    __syncthreads();
    for (int i = 0; i < 16; ++i) {
        const int at = first + w * 16 + i;
        if (at < a.words)
            a.to[which][(g * a.words + at) * 64 + lane] = tile[lane][w * 16 + i];
    }
}

template <int FA>
hipError_t few_by_b(const GemmMxArgs& a, hipStream_t st)
{
    return a.fb == kE4M3 ? few<FA, kE4M3>(a, st) : a.fb == kE5M2 ? few<FA, kE5M2>(a, st) : few<FA, kE2M1>(a, st);
}

hipError_t tiles(const MxTileArgs& x, int kind, int splits, hipStream_t st)
{
    return x.g.fa == kE4M3   ? launch_mx_tiles_e4m3(x, kind, splits, st)
           : x.g.fa == kE5M2 ? launch_mx_tiles_e5m2(x, kind, splits, st)
                             : launch_mx_tiles_e2m1(x, kind, splits, st);
}

MxPlan plan_of(const GemmMxArgs& g)
{
    return plan_gemm_mx(g.m, g.n, g.k, g.fa == kE2M1, g.fb == kE2M1, g.bf);
}

// Workspace: arranged scales of A, of B, then partial sums.
size_t arranged_bytes(int64_t rows, int64_t words) { return (size_t)(cdiv(rows, 64) * words) * 256; }

// The rows that x.g names, by one kind of tile.
hipError_t part(MxTileArgs x, int kind, int splits, hipStream_t st)
{
    x.out = splits > 1 ? kOutPart : x.g.bf ? kOutBf16 : kOutF32;
    const hipError_t e = tiles(x, kind, splits, st);
    if (e != hipSuccess || splits == 1)
        return e;
    GemmArgs j;
    j.m = x.g.m;
    j.n = x.g.n;
    j.c = x.g.c;
    j.bf = x.g.bf;
    j.acc = x.g.acc;
    j.ws = x.part;
    return launch_gemm_join(j, splits, st);
}

}  // namespace

size_t gemm_mx_workspace(const GemmMxArgs& g)
{
    if (g.k == 0)
        return 0;
    const MxPlan p = plan_of(g);
    const int64_t words = cdiv(g.k, 128);
    return (p.arranged ? arranged_bytes(g.m, words) + arranged_bytes(g.n, words) : 0) +
           (p.splits > 1 ? (size_t)p.splits * (g.m - p.main) * g.n * sizeof(float) : 0);
}

hipError_t launch_gemm_mx(const GemmMxArgs& g, hipStream_t st)
{
    if (g.k == 0) {
        GemmArgs j;
        j.m = g.m;
        j.n = g.n;
        j.c = g.c;
        j.bf = g.bf;
        j.acc = g.acc;
        return launch_gemm_join(j, 0, st);
    }
    const MxPlan p = plan_of(g);
    if (p.kind < 0)
        return g.fa == kE4M3 ? few_by_b<kE4M3>(g, st) : g.fa == kE5M2 ? few_by_b<kE5M2>(g, st) : few_by_b<kE2M1>(g, st);
    MxTileArgs x;
    x.g = g;
    x.words = (int)cdiv(g.k, 128);
    x.sa = (const uint32_t*)g.sa;
    x.sb = (const uint32_t*)g.sb;
    x.arranged = p.arranged;
    uint8_t* ws = g.ws;
    if (p.arranged) {
        ScalesArgs s;
        s.from[0] = g.sa;
        s.from[1] = g.sb;
        s.to[0] = (uint32_t*)ws;
        s.to[1] = (uint32_t*)(ws + arranged_bytes(g.m, x.words));
        s.rows[0] = g.m;
        s.rows[1] = g.n;
        s.groups_a = cdiv(g.m, 64);
        s.nb = (int)(g.k / 32);
        s.words = x.words;
        k_gemm_mx_scales<<<dim3((unsigned)(s.groups_a + cdiv(g.n, 64)), (unsigned)cdiv(x.words, 64)), kWG, 0, st>>>(s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        x.sa = s.to[0];
        x.sb = s.to[1];
        ws += arranged_bytes(g.m, x.words) + arranged_bytes(g.n, x.words);
    }
    x.part = (float*)ws;
    if (p.main == 0)
        return part(x, p.kind, p.splits, st);
    MxTileArgs rest = x;
    x.g.m = p.main;
    rest.g.m = g.m - p.main;
    rest.g.a += (g.fa == kE2M1 ? p.main * g.k / 2 : p.main * g.k);
    rest.sa += p.main * x.words;
    rest.g.sa += p.main * (g.k / 32);
    rest.g.c = (char*)g.c + p.main * g.n * (g.bf ? 2 : 4);
    const hipError_t e = part(x, 0, 1, st);
    return e == hipSuccess ? part(rest, p.kind, p.splits, st) : e;
}

}  // namespace fq
