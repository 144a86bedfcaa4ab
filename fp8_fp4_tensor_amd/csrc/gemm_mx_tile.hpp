// gemm_mx_tile.hpp -- tiles of the product of MX planes (k_gemm_mx*.hip).
//
// One workgroup computes a TM x TN tile of C, WM x WN waves of (TM/WM) x
// (TN/WN), over all of k or, where tiles are few, over a share of it (fp32
// partial sums, joined by k_gemm_join). A step is 128 bytes of a row, or with
// one 4-bit side 128 elements: rows and scales come straight from memory into
// a stage of LDS (16 or 4 bytes a lane, no registers) while the matrix unit
// works on another. Chunks of 16 bytes are permuted within a row so that 16
// lanes reading one chunk of 16 rows meet no bank twice; the transfer writes
// LDS in lane order, so it is the lane's source address that carries the
// permutation. Chunks past k read beyond the buffer's declared end, which
// gives zeros.
//
// Matrix instructions bound large products, and the clock that they leave
// (1.8 to 1.9 GHz): 8192x14336x4096 4-bit 267 us (3.6 PFLOP/s), 8-bit 382 (2.5),
// 8192x4096x14336 8-bit 356 (2.7; the library's unscaled 8-bit product of 8192^3
// reaches 2.68), 4-bit 211 (4.6). Of the 267 us 50 are stores: all workgroups end their
// tiles together. Storing a column tile just before its first product of the
// next tile only moves that wait (282 us).
#pragma once

#include "gemm_mx.hpp"
#include "mx_operand.hpp"
#include "plan.hpp"

namespace fq {
namespace {

template <int FA, int FB, bool WIDE, int TM, int TN, int WM, int WN, int NS, int S>
struct MxTile {
    static constexpr bool kBoth4 = FA == kE2M1 && FB == kE2M1;
    // Whether a workgroup takes several tiles in turn. Widened operands leave no registers for it.
    static constexpr bool kWalks = NS == 2 && !WIDE;
    static constexpr int kStep = kBoth4 ? 256 : 128;              // elements of k
    static constexpr int kRA = (int)mx_bytes<FA>(kStep), kRB = (int)mx_bytes<FB>(kStep);
    static constexpr int kNW = WM * WN, kMT = TM / WM / S, kNT = TN / WN / S;
    static constexpr int kParts = kStep / (S == 16 ? 128 : 64);   // instructions along k
    static constexpr int kIA = TM * kRA / 1024 / kNW, kIB = TN * kRB / 1024 / kNW;  // transfers of a wave
    static constexpr int kND = kStep / 128;                       // words of a row's scales
    static constexpr int kSA = (TM + 63) / 64, kSB = (TN + 63) / 64;
    static constexpr int kIS = (kND * (kSA + kSB) + kNW - 1) / kNW;
    static constexpr int kPieces = kIA + kIB + kIS;
    static_assert(TM * kRA % (1024 * kNW) == 0 && TN * kRB % (1024 * kNW) == 0, "whole transfers");
    static_assert(kPieces * (NS - 2) < 64, "outstanding transfers are counted in six bits");
    struct alignas(1024) Stage {
        uint8_t a[TM * kRA], b[TN * kRB];
        uint32_t sa[kND][kSA * 64], sb[kND][kSB * 64];
    };
};

// Which 16-byte chunk of a row of R bytes lies where.
template <int R>
__device__ __forceinline__ int chunk_at(int row, int chunk)
{
    return R == 128 ? chunk ^ (row >> 1 & 7) : chunk ^ (row >> 2 & 3);
}

// Where a lane of a transfer reads: its row of the transfer's 8 (R = 128) or 16,
// and the chunk that lies at its place, which with R = 128 depends on the
// parity of the transfer's group of 8 rows.
template <int R>
struct MxSource {
    static constexpr int kKinds = R == 128 ? 2 : 1;
    int offset[kKinds], tail[kKinds];
    __device__ __forceinline__ MxSource(int lane, int64_t bytes, int steps)
    {
        constexpr int kPer = R / 16;
#pragma unroll
        for (int q = 0; q < kKinds; ++q) {
            const int ch = chunk_at<R>(lane / kPer + 8 * q, lane % kPer);
            offset[q] = lane / kPer * (int)bytes + ch * 16;
            tail[q] = (int64_t)(steps - 1) * R + ch * 16 < bytes ? offset[q] : 0x40000000;
        }
    }
    // the transfer whose first row is `row`
    __device__ __forceinline__ int at(int row, int64_t bytes, bool last) const
    {
        const int q = kKinds == 2 ? row >> 3 & 1 : 0;
        return row * (int)bytes + (last ? tail[q] : offset[q]);
    }
};

// A lane's elements of one instruction, and its block's scale.
template <int F, bool WIDE, int S, int R>
struct MxFrag {
    i32x8 v;
    // `row`: this lane's row in LDS; chunks are numbered from the step's first
    __device__ __forceinline__ void load(const uint8_t* base, int row, int g, int part)
    {
        constexpr int G = 64 / S;
        const uint8_t* p = base + row * R;
        if constexpr (F == kE2M1) {
            const u32x4 lo = ld16(p + chunk_at<R>(row, G * part + g) * 16);
            v = join(lo, u32x4{0u, 0u, 0u, 0u});
        } else {
            const int lo = WIDE ? 2 * (G * part + g) : 2 * G * part + g, hi = WIDE ? lo + 1 : lo + G;
            v = join(ld16(p + chunk_at<R>(row, lo) * 16), ld16(p + chunk_at<R>(row, hi) * 16));
        }
    }
};

template <int FR, int FC, int S, int OPSEL>
__device__ __forceinline__ typename MxAcc<S>::T mfma_scaled(i32x8 r, uint32_t rs, i32x8 c, uint32_t cs, typename MxAcc<S>::T acc)
{
    if constexpr (S == 16)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(r, c, acc, kMfmaType<FR>, kMfmaType<FC>, OPSEL, (int)rs,
                                                                OPSEL, (int)cs);
    else
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(r, c, acc, kMfmaType<FR>, kMfmaType<FC>, OPSEL, (int)rs,
                                                               OPSEL, (int)cs);
}

// A workgroup's tiles. Workgroups go to the eight XCDs round robin and each XCD
// has its own L2, so an XCD takes a run of consecutive tiles and its workgroups
// take them in turn; runs walk down groups of eight tile rows, so that the ~32
// tiles an XCD works on at once share their rows of A and of B.
struct MxWalk {
    uint32_t at, end, step;
    __device__ __forceinline__ explicit MxWalk(uint32_t total)
    {
        const uint32_t per = total / 8, rest = total % 8, xcd = blockIdx.x % 8;
        const uint32_t start = xcd * per + min(xcd, rest);
        at = start + blockIdx.x / 8;
        end = start + per + (xcd < rest ? 1 : 0);
        step = (gridDim.x + 7) / 8;
    }
};

// `bytes` from p on, as a buffer. All lanes have the same p and bytes, which the
// compiler does not always see.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_buffer(const void* p, int bytes)
{
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// One tile's operands.
struct MxSpan {
    int64_t m0, n0;
    const uint8_t *a, *b;
    const uint32_t *sa, *sb;
    int rows_a, rows_b;  // of the tile, inside the matrices
};

// Field by field: a choice between the two in memory would put them there.
__device__ __forceinline__ MxSpan mx_pick(bool c, const MxSpan& p, const MxSpan& q)
{
    return {c ? p.m0 : q.m0, c ? p.n0 : q.n0, c ? p.a : q.a, c ? p.b : q.b, c ? p.sa : q.sa, c ? p.sb : q.sb,
            c ? p.rows_a : q.rows_a, c ? p.rows_b : q.rows_b};
}

template <int FA, int FB, int TM, int TN>
__device__ __forceinline__ MxSpan mx_span(const MxTileArgs& x, uint32_t t)
{
    const uint32_t wide = 8 * (uint32_t)x.tiles_n, band = t / wide, in = t - band * wide;
    const uint32_t high = min(8u, (uint32_t)x.tiles_m - band * 8), col = in / high;
    // the quotients are the same for all lanes, which the compiler does not see
    const uint32_t tn = __builtin_amdgcn_readfirstlane(col), tm = __builtin_amdgcn_readfirstlane(band * 8 + (in - col * high));
    MxSpan s;
    s.m0 = (int64_t)tm * TM;
    s.n0 = (int64_t)tn * TN;
    s.a = x.g.a + mx_bytes<FA>(s.m0 * x.g.k);
    s.b = x.g.b + mx_bytes<FB>(s.n0 * x.g.k);
    s.sa = x.sa + s.m0 * x.words;
    s.sb = x.sb + s.n0 * x.words;
    s.rows_a = (int)min((int64_t)TM, x.g.m - s.m0);
    s.rows_b = (int)min((int64_t)TN, x.g.n - s.n0);
    return s;
}

template <int FA, int FB, bool WIDE, int TM, int TN, int WM, int WN, int NS, int S>
__global__ __launch_bounds__(WM* WN * 64) void k_gemm_mx_tile(MxTileArgs x)
{
    using T = MxTile<FA, FB, WIDE, TM, TN, WM, WN, NS, S>;
    using Acc = typename MxAcc<S>::T;
    constexpr int MT = T::kMT, NT = T::kNT, IA = T::kIA, IB = T::kIB, IS = T::kIS, P = T::kParts, G = 64 / S;
    constexpr bool kHalves = NS == 2;
    constexpr int H = NT / 2;
    // Whether the scheduler is kept within a column tile. With widened operands beside a 64x128 tile's sums it would read
    // more of them ahead than fit the registers (14336x4096x8192: 708 us, 761 without); without either it does better
    // on its own (8192x14336x4096, 8-bit: 379 us, 389 with; 1003x7168x2048 21.3 and 21.8).
    constexpr bool kFence = WIDE && (TM / WM) * (TN / WN) >= 64 * 128;
    static_assert(!kHalves || (NT % 2 == 0 && NT >= 4 && IB % 2 == 0), "two halves of a step");
    const GemmMxArgs& g = x.g;
    __shared__ typename T::Stage stage[NS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane % S, grp = lane / S;
    MxWalk walk((uint32_t)x.tiles_m * (uint32_t)x.tiles_n);
    MxSpan span = mx_span<FA, FB, TM, TN>(x, walk.at);
    const int64_t ka = mx_bytes<FA>(g.k), kb = mx_bytes<FB>(g.k);  // bytes of a row
    const int steps = (int)((g.k + T::kStep - 1) / T::kStep);
    const int first = __builtin_amdgcn_readfirstlane((int)((int64_t)steps * blockIdx.y / gridDim.y));
    const int last = __builtin_amdgcn_readfirstlane((int)((int64_t)steps * (blockIdx.y + 1) / gridDim.y));
    // Source offsets. What lies past the last row, or past k in the last step,
    // is past any buffer (of at most 2^30 bytes) and arrives as zeros.
    constexpr int kPast = 0x40000000;
    constexpr int kRowsA = 1024 / T::kRA, kRowsB = 1024 / T::kRB;  // rows of a transfer
    const MxSource<T::kRA> src_a(lane, ka, steps);
    const MxSource<T::kRB> src_b(lane, kb, steps);
    // First row of B's transfer i of this wave: with two halves, the first IB / 2 of a wave's transfers bring the rows
    // of the first NT / 2 column tiles of every wave, the others the rest.
    auto row_b = [&](int i) {
        if constexpr (!kHalves)
            return (w * IB + i) * kRowsB;
        constexpr int kHalf = TN / WN / 2;  // rows of a wave's half
        const int at = (w * (IB / 2) + i % (IB / 2)) * kRowsB;
        return at / kHalf * 2 * kHalf + i / (IB / 2) * kHalf + at % kHalf;
    };
    // bytes between a row's words, and between rows of a group of 64
    const int scale_word = x.arranged ? 256 : 4, scale_lane = x.arranged ? 4 : x.words * 4;
    int zero = 0;  // in a register
    asm volatile("" : "+s"(zero));
    const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)stage;
    // Part of the transfer of step b into a stage: B's rows, the scales, A's rows.
    auto fill = [&](int which, const MxSpan& from, int b, int piece) {
        const uint32_t to = at + which * (uint32_t)sizeof(typename T::Stage);
        const bool tail = b == steps - 1;
        if (piece < IB) {
            const __amdgpu_buffer_rsrc_t rb = mx_buffer(from.b, (int)(from.rows_b * kb));
            to_lds<16>(rb, to + offsetof(typename T::Stage, b) + row_b(piece) * T::kRB, src_b.at(row_b(piece), kb, tail), b * T::kRB);
        } else if (piece < IB + IS) {
            // a wave brings 64 rows' words; a wave that is left over repeats a transfer, so that all count the same
            int s = w + (piece - IB) * T::kNW;
            s = s < T::kND * (T::kSA + T::kSB) ? s : 0;
            const int d = s / (T::kSA + T::kSB), slot = s % (T::kSA + T::kSB);
            const bool of_a = slot < T::kSA;
            const int group = of_a ? slot : slot - T::kSA, word = b * T::kND + d;
            // groups past the last, and words past k, are past the buffer: zeros
            const int rows = of_a ? from.rows_a : from.rows_b, groups = (rows + 63) / 64;
            const bool in = word < x.words && group < groups;
            const int off = in ? group * x.words * 256 + word * scale_word + lane * scale_lane : kPast;
            const uint32_t here = (uint32_t)__builtin_amdgcn_readfirstlane(
                (int)(to + (of_a ? offsetof(typename T::Stage, sa) + d * (T::kSA * 256)
                                 : offsetof(typename T::Stage, sb) + d * (T::kSB * 256)) + group * 256));
            to_lds<4>(mx_buffer(of_a ? from.sa : from.sb, x.arranged ? groups * x.words * 256 : rows * x.words * 4), here, off, zero);
        } else {
            const int i = w * IA + piece - IB - IS;
            const __amdgpu_buffer_rsrc_t ra = mx_buffer(from.a, (int)(from.rows_a * ka));
            to_lds<16>(ra, to + i * 1024, src_a.at(i * kRowsA, ka, tail), b * T::kRA);
        }
    };
    const int wm = w / WN, wn = w % WN;
    Acc acc[NT][MT];
    auto clear = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < MT; ++u)
                acc[t][u] = Acc{};
    };

    using FragA = MxFrag<FA, WIDE, S, T::kRA>;
    using FragB = MxFrag<FB, WIDE, S, T::kRB>;
    // A row's scale words, shifted so that an instruction's byte is that of its part: with S = 16 one word a part,
    // byte 0; with S = 32 one word for two parts, bytes 0 and 2.
    // A wave's operands: A's of a whole step, B's of the column tile at hand and of the next one.
    FragA fa[MT][P];
    uint32_t sa[MT][T::kND];
    bf16x8 wa[WIDE ? MT : 1][WIDE ? P : 1][4];
    FragB fb[2][P];
    uint32_t sb[2][T::kND];
    const int a0 = wm * (TM / WM) + row, b0 = wn * (TN / WN) + row;
    constexpr int kPer = S == 32 ? 2 : 1;  // parts of a scale word
    auto load_a = [&](const typename T::Stage& s, int u) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            fa[u][p].load(s.a, a0 + u * S, grp, p);
#pragma unroll
        for (int d = 0; d < T::kND; ++d)
            sa[u][d] = s.sa[d][a0 + u * S] >> (8 * grp);
    };
    auto load_b = [&](const typename T::Stage& s, int t, int into) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            fb[into][p].load(s.b, b0 + t * S, grp, p);
#pragma unroll
        for (int d = 0; d < T::kND; ++d)
            sb[into][d] = s.sb[d][b0 + t * S] >> (8 * grp);
    };
    auto widen_a = [&]() {
        if constexpr (WIDE) {
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const float f = e8m0_value(sa[u][p / kPer] >> (p % kPer * 16) & 0xFFu);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        wa[u][p][e] = widen8<FA>(fa[u][p].v, e, f);
                }
        }
    };
    // The products of column tile t; after(u) follows the last one that reads A's row tile u.
    auto products = [&](int t, auto after) {
        const int k = t & 1;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if constexpr (WIDE) {
                const float f = e8m0_value(sb[k][p / kPer] >> (p % kPer * 16) & 0xFFu);
                bf16x8 wb[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    wb[e] = widen8<FB>(fb[k][p].v, e, f);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int u = 0; u < MT; ++u) {
                        acc[t][u] = mfma_bf16<S>(wb[e], wa[u][p][e], acc[t][u]);
                        if (p == P - 1 && e == 3)
                            after(u);
                    }
            } else {
#pragma unroll
                for (int u = 0; u < MT; ++u) {
                    if (p % kPer)
                        acc[t][u] = mfma_scaled<FB, FA, S, 2>(fb[k][p].v, sb[k][p / kPer], fa[u][p].v, sa[u][p / kPer], acc[t][u]);
                    else
                        acc[t][u] = mfma_scaled<FB, FA, S, 0>(fb[k][p].v, sb[k][p / kPer], fa[u][p].v, sa[u][p / kPer], acc[t][u]);
                    if (p == P - 1)
                        after(u);
                }
            }
        }
    };
    // Sums that are infinite or no numbers where the scales of a row of A or of B can be the cause (see add_block): they are
    // noted, left out when the others are stored, and then, when the sums' registers are free, added up again. In code of
    // its own, one sum after the other: what the ordinary way pays is a look at some sums (4096x4096x4096, 8-bit: 109.2 us,
    // 108.7 without; a branch around each store of the ordinary way would cost 1%).
    constexpr int E = S * S / 64;  // sums of a lane in an instruction's tile
    auto not_finite = [&]() {
        // An infinite value leaves no finite sum in its whole row (column): those of one column tile's first column and of one
        // row tile tell. NaN if one is not finite; four chains, for each addition waits for the one before.
        float zeros[4] = {};
#pragma unroll
        for (int u = 0; u < MT; ++u)
            zeros[u % 4] = __builtin_fmaf(acc[0][u][0], 0.0f, zeros[u % 4]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < E; ++e)
                zeros[e % 4] = __builtin_fmaf(acc[t][0][e], 0.0f, zeros[e % 4]);
        const float zero = (zeros[0] + zeros[1]) + (zeros[2] + zeros[3]);
        return __ballot(zero != 0.0f) != 0;
    };
    // Stores all sums and returns true, or false if none of the scales is that large.
    auto store_beyond = [&](const MxSpan& s) {
        // What it takes is loaded and computed here: kept since the kernel's start it would change the steps' registers and
        // with them the order of their instructions (256x4096x4096 23.1 us, 22.4 so, 22.0 without all of this).
        typedef const MxTileArgs __attribute__((address_space(4))) * Kernarg;
        Kernarg at = (Kernarg)__builtin_amdgcn_kernarg_segment_ptr();
        int thread = threadIdx.x;
        asm volatile("" : "+s"(at), "+v"(thread));
        const uint8_t *ga = at->g.a, *gb = at->g.b, *gsa = at->g.sa, *gsb = at->g.sb;
        const int64_t m = at->g.m, n = at->g.n, k = at->g.k, nb = k >> 5;
        const bool part = at->out == kOutPart, add = !part && at->g.acc;
        float* const to = part ? at->part + (int64_t)blockIdx.y * m * n : (float*)at->g.c;
        const int lane = thread & 63, w = __builtin_amdgcn_readfirstlane(thread >> 6), row = lane % S, grp = lane / S;
        const int64_t i0 = s.m0 + w / WN * (TM / WM), j0 = s.n0 + w % WN * (TN / WN);
        const int64_t block0 = (int64_t)first * (T::kStep / 32), block1 = min((int64_t)last * (T::kStep / 32), nb);
        // this lane's row of row tile u of A, of column tile t of B; rows past the last repeat it and are not stored
        auto row_of_a = [&](int u) { return min(i0 + u * S + row, m - 1); };
        auto row_of_b = [&](int t) { return min(j0 + t * S + row, n - 1); };
        uint32_t far_a = 0, far_b = 0;  // a bit for each of this lane's rows
#pragma unroll 1
        for (int u = 0; u < MT; ++u)
            far_a |= past_top<FA, S>(gsa + row_of_a(u) * nb, block0, block1, grp) ? 1u << u : 0u;
#pragma unroll 1
        for (int t = 0; t < NT; ++t)
            far_b |= past_top<FB, S>(gsb + row_of_b(t) * nb, block0, block1, grp) ? 1u << t : 0u;
        if (__ballot((far_a | far_b) != 0) == 0)
            return false;
        auto put_one = [&](int t, int u, int e, float v) {
            const int64_t i = i0 + u * S + row, j = j0 + t * S + row_of_sum<S>(e, grp);
            if (i < m && j < n)
                to[i * n + j] = add ? to[i * n + j] + v : v;
        };
        constexpr int kWords = (NT * MT * E + 31) / 32;
        uint32_t again[kWords] = {};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t far = far_a >> u | __shfl(far_b, row_of_sum<S>(e, grp)) >> t;
                    const int bit = (t * MT + u) * E + e;
                    if ((far & 1) && no_number(acc[t][u][e]))
                        again[bit / 32] |= 1u << bit % 32;
                    else
                        put_one(t, u, e, acc[t][u][e]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll 1
        for (int q = 0; q < NT * MT; ++q) {
            uint32_t bits = 0;
#pragma unroll
            for (int y = 0; y < kWords; ++y)
                bits = q * E / 32 == y ? again[y] >> q * E % 32 : bits;
            bits &= (1u << E) - 1;
            if (__ballot(bits != 0) == 0)
                continue;
            const int64_t i = row_of_a(q % MT), j = row_of_b(q / MT);
            const uint8_t *pa = ga + mx_bytes<FA>(i * k), *pb = gb + mx_bytes<FB>(j * k);
            Acc sum{};
#pragma unroll 1
            for (int64_t b = block0; b < block1; ++b)
                add_block<FA, FB, S>(pa, gsa + i * nb, pb, gsb + j * nb, b, grp, sum);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (bits >> e & 1)
                    put_one(q / MT, q % MT, e, sum[e]);
        }
        return true;
    };
    auto store = [&](const MxSpan& s) {
        // A lane has, of row i, four consecutive columns from 4 grp on (S = 16), or four from 8 q + 4 grp on for q < 4.
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int64_t i = s.m0 + wm * (TM / WM) + u * S + row;
            const int64_t j0 = s.n0 + wn * (TN / WN);
            if (x.out == kOutBf16 && (g.n & 7) == 0) {
                // Exchanging between lane groups leaves eight consecutive columns in a lane.
                constexpr int Q = S == 16 ? 1 : 4;
                if constexpr (S == 32 || NT % 2 == 0) {
#pragma unroll
                    for (int t = 0; t < NT * Q; t += 2) {
                        auto four = [&](int q) {
                            if constexpr (S == 16)
                                return acc[q][u];
                            else
                                return f32x4{acc[q / 4][u][q % 4 * 4], acc[q / 4][u][q % 4 * 4 + 1], acc[q / 4][u][q % 4 * 4 + 2],
                                             acc[q / 4][u][q % 4 * 4 + 3]};
                        };
                        const f32x4 lo = four(t), hi = four(t + 1);
                        uint32_t w0[2], w1[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t p = bf16_bits(lo[2 * e]) | bf16_bits(lo[2 * e + 1]) << 16;
                            const uint32_t q = bf16_bits(hi[2 * e]) | bf16_bits(hi[2 * e + 1]) << 16;
                            const u32x2 r = __builtin_bit_cast(u32x2, S == 16 ? __builtin_amdgcn_permlane16_swap(p, q, false, false)
                                                                              : __builtin_amdgcn_permlane32_swap(p, q, false, false));
                            w0[e] = r[0];
                            w1[e] = r[1];
                        }
                        const int64_t j = S == 16 ? j0 + (t + (grp & 1)) * 16 + (grp >> 1) * 8 : j0 + (t + grp) * 8;
                        if (i < g.m && j < g.n)
                            *(u32x4*)((uint16_t*)g.c + i * g.n + j) = u32x4{w0[0], w0[1], w1[0], w1[1]};
                    }
                    continue;
                }
            }
            if (i < g.m) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int q = 0; q < S / 4 / G; ++q) {
                        const int64_t j = j0 + t * S + q * 8 + grp * 4;
                        f32x4 v;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = acc[t][u][q * 4 + e];
                        if (x.out == kOutPart)
                            store4<false>(x.part + (int64_t)blockIdx.y * g.m * g.n, i, j, g.n, v, false);
                        else if (x.out == kOutBf16)
                            store4<true>(g.c, i, j, g.n, v, false);
                        else
                            store4<false>(g.c, i, j, g.n, v, g.acc);
                    }
            }
        }
    };
    auto put = [&](const MxSpan& s) {
        if constexpr (WIDE)
            if (__builtin_expect(not_finite(), 0) && store_beyond(s))
                return;
        store(s);
    };
    if constexpr (kHalves) {
        // Steps run on from one tile to the next. A step's last products
        // overlap the reads of the next one's first operands, so the two
        // barriers of a step stand one column tile ahead of what they guard,
        // and every transfer has a step or more to arrive, in the order of its need:
        //   first half of step b    the second half of B(b + 1), after the barrier that ended its use
        //   barrier                 the second half of B(b) has arrived; A(b) is in registers, the first half of B(b) read
        //   second half             A(b + 2) and the first half of B(b + 2), over those of b
        //   barrier                 A(b + 1), its scales and the first half of B(b + 1) have arrived; B(b) has been read
        // The scales of b + 1 go first in the first half. Behind the last tile
        // the last step is fetched again, unused: without branches the step is one run of code.
        auto scales_b2 = [&](int which, const MxSpan& from, int b, int i) { fill(which, from, b, i < IS ? IB + i : IB / 2 + i - IS); };
        auto a_b1 = [&](int which, const MxSpan& from, int b, int i) { fill(which, from, b, i < IA ? IB + IS + i : i - IA); };
        constexpr int N1 = IS + IB / 2, N2 = IA + IB / 2;
#pragma unroll
        for (int i = 0; i < IS; ++i)
            fill(0, span, first, IB + i);
#pragma unroll
        for (int i = 0; i < N2; ++i)
            a_b1(0, span, first, i);
#pragma unroll
        for (int i = 0; i < IB / 2; ++i)
            fill(0, span, first, IB / 2 + i);
#pragma unroll
        for (int i = 0; i < N2; ++i)
            a_b1(1, span, min(first + 1, last - 1), i);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(IA + IB) : "memory");
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MT; ++u)
            load_a(stage[0], u);
        load_b(stage[0], 0, 0);
        int here = 0;
        for (;;) {
            walk.at += walk.step;
            const bool more = T::kWalks && walk.at < walk.end;
            const MxSpan next = more ? mx_span<FA, FB, TM, TN>(x, walk.at) : span;
            clear();
            for (int b = first; b < last; ++b, here ^= 1) {
                const typename T::Stage &s = stage[here], &n = stage[here ^ 1];
                // the steps that are fetched: of this tile, or the next one's first (a tile has two steps at least then)
                const bool in1 = b + 1 < last || !more, in2 = b + 2 < last || !more;
                const MxSpan from1 = mx_pick(in1, span, next), from2 = mx_pick(in2, span, next);
                const int b1 = in1 ? min(b + 1, last - 1) : first, b2 = in2 ? min(b + 2, last - 1) : first + b + 2 - last;
                widen_a();
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t + 1 < NT) {
                        load_b(s, t + 1, (t + 1) & 1);
                        products(t, [](int) {});
                    } else {
                        load_b(n, 0, 0);
                        products(t, [&](int u) { load_a(n, u); });
                    }
                    if constexpr (kFence)
                        __builtin_amdgcn_sched_barrier(0);
                    if (t < H - 1) {
#pragma unroll
                        for (int i = t * N1 / (H - 1); i < (t + 1) * N1 / (H - 1); ++i)
                            scales_b2(here ^ 1, from1, b1, i);
                    } else if (t < NT - 1) {
#pragma unroll
                        for (int i = (t - H + 1) * N2 / H; i < (t - H + 2) * N2 / H; ++i)
                            a_b1(here, from2, b2, i);
                    }
                    if (t == H - 2)
                        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(IA + IB + IS) : "memory");
                    if (t == NT - 2)
                        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(IA + IB) : "memory");
                }
            }
            put(span);
            if (!more)
                break;
            span = next;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    } else {
        clear();
#pragma unroll
        for (int p = 0; p < NS - 1; ++p)
            if (first + p < last) {
#pragma unroll
                for (int i = 0; i < T::kPieces; ++i)
                    fill(p, span, first + p, i);
            }
        int here = 0, there = NS - 1;
        for (int b = first; b < last; ++b) {
            if (b + NS - 1 <= last)  // NS - 1 steps are under way: all but the oldest may stay so
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(T::kPieces*(NS - 2)) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (b + NS - 1 < last) {
#pragma unroll
                for (int i = 0; i < T::kPieces; ++i)
                    fill(there, span, b + NS - 1, i);
            }
#pragma unroll
            for (int u = 0; u < MT; ++u)
                load_a(stage[here], u);
            load_b(stage[here], 0, 0);
            widen_a();
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t + 1 < NT)
                    load_b(stage[here], t + 1, (t + 1) & 1);
                products(t, [](int) {});
                // keeps the scheduler from reading all operands at once, which would not fit the registers
                __builtin_amdgcn_sched_barrier(0);
            }
            here = here + 1 == NS ? 0 : here + 1;
            there = there + 1 == NS ? 0 : there + 1;
        }
        put(span);
    }
}

template <int FA, int FB, bool WIDE, int TM, int TN, int WM, int WN, int NS, int S>
hipError_t mx_run(MxTileArgs x, int splits, hipStream_t st)
{
    x.tiles_m = (int)cdiv(x.g.m, TM);
    x.tiles_n = (int)cdiv(x.g.n, TN);
    const int64_t tiles = (int64_t)x.tiles_m * x.tiles_n;
    using T = MxTile<FA, FB, WIDE, TM, TN, WM, WN, NS, S>;
    // a workgroup a CU walks, if a tile has the two steps that are under way
    const bool walks = T::kWalks && splits == 1 && x.g.k > T::kStep && tiles > kChipCus;
    k_gemm_mx_tile<FA, FB, WIDE, TM, TN, WM, WN, NS, S>
        <<<dim3((unsigned)(walks ? kChipCus : tiles), (unsigned)splits), WM * WN * 64, 0, st>>>(x);
    return hipGetLastError();
}

template <int FA, int FB, bool WIDE>
hipError_t mx_tiles(const MxTileArgs& x, int kind, int splits, hipStream_t st)
{
    switch (kind) {
    case 0: return mx_run<FA, FB, WIDE, kMxTiles[0].tm, kMxTiles[0].tn, 4, 2, 2, 32>(x, splits, st);
    case 1: return mx_run<FA, FB, WIDE, kMxTiles[1].tm, kMxTiles[1].tn, 2, 4, 2, 16>(x, splits, st);
    case 2: return mx_run<FA, FB, WIDE, kMxTiles[2].tm, kMxTiles[2].tn, 1, 4, 3, 16>(x, splits, st);
    default: return mx_run<FA, FB, WIDE, kMxTiles[3].tm, kMxTiles[3].tn, 1, 4, 3, 16>(x, splits, st);
    }
}

// A's format fixed, B's and the result's by the call.
template <int FA>
hipError_t mx_launch(const MxTileArgs& x, int kind, int splits, hipStream_t st)
{
    const bool f32 = !x.g.bf;
    switch (x.g.fb) {
    case kE4M3: return f32 ? mx_tiles<FA, kE4M3, true>(x, kind, splits, st) : mx_tiles<FA, kE4M3, false>(x, kind, splits, st);
    case kE5M2: return f32 ? mx_tiles<FA, kE5M2, true>(x, kind, splits, st) : mx_tiles<FA, kE5M2, false>(x, kind, splits, st);
    default:
        if (kWidened<FA, kE2M1, true> && f32)
            return mx_tiles<FA, kE2M1, kWidened<FA, kE2M1, true>>(x, kind, splits, st);
        return mx_tiles<FA, kE2M1, false>(x, kind, splits, st);
    }
}

}  // namespace
}  // namespace fq
