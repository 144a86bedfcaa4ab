// k_gemm.hip -- the matrix product of blockwise-scaled E4M3 planes on gfx950.
//
//   C[i, j] = sum_b sa[i, b] * sb[j, b] * sum_{t < 128} A[i, 128 b + t] * B[j, 128 b + t]
//
// A: [m, k] codes with 1x128 scales; B: [n, k] codes with 128x128 scales
// (one scale row for 128 rows of B) or 1x128 scales. Both operands run along
// k, so a 128-byte run of a row is one scale block, one cache line and the
// whole depth of one v_mfma_f32_16x16x128_f8f6f4: the instruction's result
// from a zero accumulator is the inner sum of one block, and one fused
// multiply-add per value adds it, scaled, to the running fp32 sum.
//
// Two ways to the inner sum. The 8-bit instruction aligns the products of a
// sum before it adds them and keeps few bits below the largest: measured over
// 4096 tiles, a block's sum is off by up to 6e-4 of its largest product, 1.3e-5
// (normal values) to 5e-5 (values over 16 binades) of the result in the mean
// square. Next to a bf16 output's own rounding (1.7e-3) that is nothing, and it
// is the full rate of the matrix unit. An fp32 output gets sums that are fp32
// throughout: the codes become bf16 (exact) and meet in four
// v_mfma_f32_16x16x32_bf16, off by 1e-8, at half the rate.
//
// Operand order: B's rows are the instruction's rows and A's rows its
// columns, so a lane holds one row i of C and four consecutive columns j:
// its 128x128-scaled multiplier is ONE value, sa[i, b] * sb[b], and its four
// results are one contiguous store. Lane l supplies row l % 16 of either
// operand and, of its 128-byte run, the 16-byte chunks l / 16 and 4 + l / 16
// (any assignment of the depth serves, the same for both operands).
#include "codec.hpp"
#include "launch.hpp"
#include "plan.hpp"

namespace fq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight E4M3 codes -> eight bf16 (exact).
__device__ __forceinline__ bf16x8 widen8(int a, int b)
{
    const bf16x2 r0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)a, 1.0f, false);
    const bf16x2 r1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)a, 1.0f, true);
    const bf16x2 r2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)b, 1.0f, false);
    const bf16x2 r3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)b, 1.0f, true);
    return bf16x8{r0[0], r0[1], r1[0], r1[1], r2[0], r2[1], r3[0], r3[1]};
}

// The inner sum of one scale block for 16x16 outputs.
template <bool BF>
__device__ __forceinline__ f32x4 mfma_block(i32x8 rows, i32x8 cols)
{
    const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (!BF) {
        f32x4 c = z;
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(rows[e], rows[e + 1]), widen8(cols[e], cols[e + 1]), c,
                                                        0, 0, 0);
        return c;
    }
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(rows, cols, z, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi)
{
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ uint32_t bf16_bits(float v)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// Four consecutive outputs C[i, j .. j+3] of a row; those at or past n are not written.
template <bool BF>
__device__ __forceinline__ void store4(void* c, int64_t i, int64_t j, int64_t n, f32x4 v, bool acc)
{
    if constexpr (BF) {
        uint16_t* p = (uint16_t*)c + i * n + j;
        if ((n & 3) == 0) {
            if (j < n)
                *(u32x2*)p = u32x2{bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < n)
                p[e] = (uint16_t)bf16_bits(v[e]);
    } else {
        float* p = (float*)c + i * n + j;
        if ((n & 3) == 0) {
            if (j < n) {
                if (acc)
                    v += *(const f32x4*)p;
                *(f32x4*)p = v;
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < n)
                p[e] = acc ? p[e] + v[e] : v[e];
    }
}

// Few rows of A (m <= 16) and no more columns than the chip holds at once: one
// workgroup computes 16 columns; its waves take the blocks of k in turn and
// their sums meet in LDS, in wave order. Nothing is reused but A (from L2),
// so operands go straight from memory to the matrix unit's registers; the
// loads of 32 waves a CU hide each other's latency (a block fetched ahead in
// registers measured slower: 6.6 us for 1x4096x4096 against 5.4).
constexpr int kFewWaves = 8;

template <bool B1, bool BF>
__global__ __launch_bounds__(kFewWaves * 64) void k_gemm_few(GemmArgs g)
{
    __shared__ f32x4 part[kFewWaves][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = lane & 15, grp = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int nb = (int)(g.k >> 7);
    // rows and columns past the last repeat it and are not stored
    const int64_t i = min((int64_t)row, g.m - 1), j = min(n0 + row, g.n - 1);
    const uint8_t* pa = g.a + i * g.k + grp * 16;
    const uint8_t* pb = g.b + j * g.k + grp * 16;
    const float* psa = g.sa + i * nb;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = w; b < nb; b += kFewWaves) {
        const i32x8 fb = join(ld16_stream(pb + (int64_t)b * 128), ld16_stream(pb + (int64_t)b * 128 + 64));
        const i32x8 fa = join(ld16(pa + (int64_t)b * 128), ld16(pa + (int64_t)b * 128 + 64));
        const float sa = psa[b];
        float sb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sb[e] = B1 ? g.sb[min(n0 + grp * 4 + e, g.n - 1) * nb + b] : g.sb[(n0 >> 7) * nb + b];
        const f32x4 p = mfma_block<BF>(fb, fa);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[e] = __builtin_fmaf(p[e], sa * sb[e], acc[e]);
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w > 0 || row >= g.m)
        return;
#pragma unroll
    for (int x = 1; x < kFewWaves; ++x)
        acc += part[x][lane];
    store4<BF>(g.c, row, n0 + grp * 4, g.n, acc, g.acc);
}

hipError_t few(const GemmArgs& g, hipStream_t st)
{
    const dim3 grid((unsigned)cdiv(g.n, 16));
    constexpr int th = kFewWaves * 64;
    if (g.b1)
        g.bf ? k_gemm_few<true, true><<<grid, th, 0, st>>>(g) : k_gemm_few<true, false><<<grid, th, 0, st>>>(g);
    else
        g.bf ? k_gemm_few<false, true><<<grid, th, 0, st>>>(g) : k_gemm_few<false, false><<<grid, th, 0, st>>>(g);
    return hipGetLastError();
}

// ---------------------------------------------------------------- tiles
// One workgroup computes a TM x TN tile of C, WM x WN waves of
// (TM/WM) x (TN/WN), over all blocks of k or, where tiles are few, over a
// share of them (SPLIT: fp32 partial sums, joined by k_gemm_join). A step is
// one scale block: TM + TN rows of 128 bytes come straight from memory into
// one of NS stages of LDS (16 bytes a lane, no registers), NS - 1 steps ahead
// of the products. The 16-byte chunk c of row r is kept at chunk c ^ (r % 8)
// of its row, so that eight lanes reading one chunk of eight rows meet no bank
// twice; the transfer writes LDS in lane order, so it is the lane's source
// address that carries the permutation.

// 64 lanes' 16 (or 4) bytes each -> LDS at `to`, in lane order. Written as
// assembly because the compiler, which cannot tell the two stages apart,
// would wait for every transfer before the next read of LDS; there is no
// output register, and the waits are those of the step loop. M0 holds the
// LDS address and needs one wait state before its use; naming it as written
// keeps the compiler's own uses of it apart (it warns of any reserved register
// in that list).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, uint32_t to, int lane_offset, int offset)
{
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :
                     : "s"(to), "v"(lane_offset), "s"(r), "s"(offset)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                     :
                     : "s"(to), "v"(lane_offset), "s"(r), "s"(offset)
                     : "memory", "m0");
}
#pragma clang diagnostic pop

// Workgroup -> tile. Workgroups go to the eight XCDs round robin and each XCD
// has its own L2, so an XCD takes a run of consecutive tiles; runs walk down
// groups of eight tile rows, so the ~32 tiles an XCD works on at once share
// their rows of A and of B.
__device__ __forceinline__ void tile_of(const GemmArgs& g, int64_t& tm, int64_t& tn)
{
    const uint32_t total = gridDim.x, per = total / 8, rest = total % 8;
    const uint32_t xcd = blockIdx.x % 8, nth = blockIdx.x / 8;
    const uint32_t t = xcd * per + min(xcd, rest) + nth;
    const uint32_t wide = 8 * (uint32_t)g.tiles_n;
    const uint32_t band = t / wide, in = t - band * wide;
    const uint32_t high = min(8u, (uint32_t)g.tiles_m - band * 8);
    tn = in / high;
    tm = band * 8 + (in - (uint32_t)tn * high);
}

template <int TM, int TN, int WM, int WN, int NS, bool B1>
struct Tile {
    static constexpr int kNW = WM * WN;
    static constexpr int kMT = TM / WM / 16, kNT = TN / WN / 16;
    static_assert(B1 || TN / WN <= 128, "a wave's columns share a 128x128 scale");
    // transfers a wave issues for a step: eight rows each, and 64 scales
    static constexpr int kIA = TM / 8 / kNW, kIB = TN / 8 / kNW, kPieces = kIA + kIB + 1;
    static constexpr int kSA = (TM + 63) / 64, kSB = B1 ? TN / 64 : 1;
    static_assert(TM % (8 * kNW) == 0 && TN % (8 * kNW) == 0, "whole transfers");
    static_assert(kNW >= kSA + kSB, "a wave brings 64 scales");
    static_assert(kPieces * (NS - 2) < 64, "outstanding transfers are counted in six bits");
    struct alignas(1024) Stage {
        uint8_t a[TM * 128], b[TN * 128];
        float sa[kSA * 64], sb[kSB * 64];
    };
};

template <int TM, int TN, int WM, int WN, int NS, bool SPLIT, bool B1, bool BF>
__global__ __launch_bounds__(WM* WN * 64) void k_gemm_tile(GemmArgs g)
{
    using T = Tile<TM, TN, WM, WN, NS, B1>;
    // both stages full and few reads of A: see the step
    constexpr bool kLateA = NS == 2 && T::kNT == 8 && T::kIA <= 4;
    constexpr int MT = T::kMT, NT = T::kNT, IA = T::kIA, IB = T::kIB, kPieces = T::kPieces;
    __shared__ typename T::Stage stage[NS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, grp = lane >> 4;
    int64_t tm, tn;
    tile_of(g, tm, tn);
    const int64_t m0 = tm * TM, n0 = tn * TN;
    const int nb = (int)(g.k >> 7);
    // this workgroup's blocks of k: [first, last)
    const int first = SPLIT ? (int)((int64_t)nb * blockIdx.y / gridDim.y) : 0;
    const int last = SPLIT ? (int)((int64_t)nb * (blockIdx.y + 1) / gridDim.y) : nb;
    const int rows_a = (int)min((int64_t)TM, g.m - m0), rows_b = (int)min((int64_t)TN, g.n - n0);
    const uint8_t* pa = g.a + m0 * g.k;
    const uint8_t* pb = g.b + n0 * g.k;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)pa, 0, (int)(rows_a * g.k), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)pb, 0, (int)(rows_b * g.k), 0x00020000);
    // the scales of one block: the first waves bring A's, the next ones B's;
    // a wave that is left over repeats a transfer, so that all count the same
    const bool of_a = w < T::kSA;
    const int slot = of_a ? w : w < T::kSA + T::kSB ? w - T::kSA : 0;
    const int rows_s = of_a ? rows_a : B1 ? rows_b : (rows_b + 127) >> 7;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(of_a ? g.sa + m0 * nb : g.sb + (B1 ? n0 : n0 >> 7) * nb), 0, rows_s * nb * 4, 0x00020000);
    // rows past the last repeat it, so every source address is inside; they are not stored
    int va[IA], vb[IB];
    const int sub = lane >> 3, chunk = (lane & 7) ^ sub;
#pragma unroll
    for (int i = 0; i < IA; ++i)
        va[i] = min((w * IA + i) * 8 + sub, rows_a - 1) * (int)g.k + chunk * 16;
#pragma unroll
    for (int i = 0; i < IB; ++i)
        vb[i] = min((w * IB + i) * 8 + sub, rows_b - 1) * (int)g.k + chunk * 16;
    const int vs = min(slot * 64 + lane, rows_s - 1) * nb * 4;
    const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)stage;
    // Part of the transfer of block b into a stage: `piece` 0 .. IA + IB - 1
    // is eight rows of B or A, the last one the scales.
    auto fill = [&](int which, int b, int piece) {
        const uint32_t to = at + which * (uint32_t)sizeof(typename T::Stage);
        if (piece < IB)
            to_lds<16>(rb, to + offsetof(typename T::Stage, b) + (w * IB + piece) * 1024, vb[piece < IB ? piece : 0], b * 128);
        else if (piece < IB + IA)
            to_lds<16>(ra, to + (w * IA + piece - IB) * 1024, va[piece - IB < IA ? piece - IB : 0], b * 128);
        else
            to_lds<4>(rs, to + (of_a ? offsetof(typename T::Stage, sa) : offsetof(typename T::Stage, sb)) + slot * 256, vs,
                      b * 4);
    };
    const int wm = w / WN, wn = w % WN;
    const int c0 = ((grp ^ (row & 7)) * 16), c1 = c0 ^ 64;
    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
            acc[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto work = [&](const typename T::Stage& s, int which, int next, int after) {
        i32x8 fa[MT];
        float sc[MT];
        const float sbv = s.sb[wn * (TN / WN) / 128];  // 128x128 tiles: one scale for the wave's columns
        const uint8_t* qa = s.a + (wm * (TM / WM) + row) * 128;
        const uint8_t* qb = s.b + (wn * (TN / WN) + row) * 128;
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            fa[u] = join(ld16(qa + u * 2048 + c0), ld16(qa + u * 2048 + c1));
            sc[u] = s.sa[wm * (TM / WM) + u * 16 + row];
            if constexpr (!B1)
                sc[u] *= sbv;
        }
        // The next column tile's operand is read during this one's products.
        // The fences keep the scheduler from reading all of them at once,
        // which would not fit the registers. The next block's transfers go out
        // between them: all at once, their issue holds up this step's reads of
        // LDS (8192x4096x14336 with 256x256 tiles: 493 us; spread over half of
        // the step 455, the whole step 482, for they arrive late; A a step
        // earlier 409).
        i32x8 fb = join(ld16(qb + c0), ld16(qb + c1));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            i32x8 nx = fb;
            if (t + 1 < NT)
                nx = join(ld16(qb + (t + 1) * 2048 + c0), ld16(qb + (t + 1) * 2048 + c1));
            f32x4 sb4;
            if constexpr (B1)
                sb4 = *(const f32x4*)&s.sb[wn * (TN / WN) + t * 16 + grp * 4];
#pragma unroll
            for (int u = 0; u < MT; ++u) {
                const f32x4 p = mfma_block<BF>(fb, fa[u]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[t][u][e] = __builtin_fmaf(p[e], B1 ? sc[u] * sb4[e] : sc[u], acc[t][u][e]);
            }
            fb = nx;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (kLateA) {
                // B and the scales of the next block first, two pieces a tile;
                // half way every wave holds its part of A in registers, so that
                // the A of the block after that can replace it already: a
                // step and a half to arrive, where the whole of a block
                // brought at once has one
                if (t * 2 < IB + 1)
                    fill(which, next, t * 2 < IB ? t * 2 : IA + IB);
                if (t * 2 + 1 < IB + 1)
                    fill(which, next, t * 2 + 1 < IB ? t * 2 + 1 : IA + IB);
                if (t == NT / 2)
                    asm volatile("s_barrier" ::: "memory");
                if (t >= NT / 2 && t - NT / 2 < IA)
                    fill(which ^ 1, after, IB + t - NT / 2);
            } else if constexpr (NS == 2) {
#pragma unroll
                for (int i = min(2 * t * kPieces / NT, kPieces); i < min(2 * (t + 1) * kPieces / NT, kPieces); ++i)
                    fill(which, next, i);
            }
        }
    };
    // Each wave waits for its own transfers of the step before the barrier;
    // after it the step's stage is whole, and every wave has read the stage
    // that the next transfers overwrite.
    if constexpr (NS == 2) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            fill(0, first, i);
        if constexpr (kLateA) {
#pragma unroll
            for (int i = 0; i < IA; ++i)
                fill(1, min(first + 1, last - 1), IB + i);
        }
        for (int b = first; b < last; ++b) {
            // with kLateA all but the A of the block after next, which went out last
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLateA ? IA : 0) : "memory");
            __syncthreads();
            // the last steps fetch their own block again, unused: without
            // branches the step is one run of code
            work(stage[(b - first) & 1], (b - first + 1) & 1, min(b + 1, last - 1), min(b + 2, last - 1));
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    } else {
#pragma unroll
        for (int p = 0; p < NS - 1; ++p)
            if (first + p < last) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    fill(p, first + p, i);
            }
        int here = 0, there = NS - 1;
        for (int b = first; b < last; ++b) {
            if (b + NS - 1 <= last)  // NS - 1 blocks are under way: all but the oldest may stay so
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kPieces*(NS - 2)) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (b + NS - 1 < last) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    fill(there, b + NS - 1, i);
            }
            work(stage[here], 0, 0, 0);
            here = here + 1 == NS ? 0 : here + 1;
            there = there + 1 == NS ? 0 : there + 1;
        }
    }
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const int64_t i = m0 + wm * (TM / WM) + u * 16 + row;
        if constexpr (BF && !SPLIT && NT % 2 == 0) {
            // Two column tiles at once: exchanging odd lane groups of the one
            // with even groups of the other leaves eight consecutive columns in
            // a lane, 64 bytes of a row in an instruction (8192x14336x4096:
            // 452 us, 474 with 32 bytes of a row; 1003x7168x2048: 22.9, 24.7).
            if ((g.n & 7) == 0) {
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t w0[2], w1[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t x = bf16_bits(acc[t][u][2 * e]) | bf16_bits(acc[t][u][2 * e + 1]) << 16;
                        const uint32_t y = bf16_bits(acc[t + 1][u][2 * e]) | bf16_bits(acc[t + 1][u][2 * e + 1]) << 16;
                        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, y, false, false));
                        w0[e] = r[0];
                        w1[e] = r[1];
                    }
                    const int64_t j = n0 + wn * (TN / WN) + (t + (grp & 1)) * 16 + (grp >> 1) * 8;
                    if (i < g.m && j < g.n)
                        *(u32x4*)((uint16_t*)g.c + i * g.n + j) = u32x4{w0[0], w0[1], w1[0], w1[1]};
                }
                continue;
            }
        }
        if (i < g.m)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int64_t j = n0 + wn * (TN / WN) + t * 16 + grp * 4;
                if constexpr (SPLIT)
                    store4<false>(g.ws + (int64_t)blockIdx.y * g.m * g.n, i, j, g.n, acc[t][u], false);
                else
                    store4<BF>(g.c, i, j, g.n, acc[t][u], g.acc);
            }
    }
}

// C = the sum of the splits' partial results, in their order (zeros for k = 0,
// which has none); four values a thread.
template <bool BF>
__global__ __launch_bounds__(kWG) void k_gemm_join(GemmArgs g, int splits)
{
    const int64_t total = g.m * g.n;
    const int64_t e = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWG + threadIdx.x) * 4;
    if (e >= total)
        return;
    if (total % 4) {  // partial results are not 16-byte aligned
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (e + i >= total)
                return;
            float v = 0.0f;
            for (int s = 0; s < splits; ++s)
                v += g.ws[s * total + e + i];
            if constexpr (BF)
                ((uint16_t*)g.c)[e + i] = (uint16_t)bf16_bits(v);
            else
                ((float*)g.c)[e + i] = g.acc ? ((float*)g.c)[e + i] + v : v;
        }
        return;
    }
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < splits; ++s)
        v += *(const f32x4*)(g.ws + s * total + e);
    store4<BF>(g.c, 0, e, total, v, g.acc);
}

hipError_t join(const GemmArgs& g, int splits, hipStream_t st)
{
    // at most 2^26 workgroups; a grid's dimension has less than 2^32 threads
    const int64_t need = cdiv(cdiv(g.m * g.n, 4), kWG), across = need < (1 << 23) ? need : 1 << 23;
    const dim3 blocks((unsigned)across, (unsigned)cdiv(need, across));
    g.bf ? k_gemm_join<true><<<blocks, kWG, 0, st>>>(g, splits) : k_gemm_join<false><<<blocks, kWG, 0, st>>>(g, splits);
    return hipGetLastError();
}

template <int TM, int TN, int WM, int WN, int NS, bool SPLIT>
hipError_t run_tiles(const GemmArgs& g, int splits, hipStream_t st)
{
    const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n), (unsigned)splits);
    constexpr int th = WM * WN * 64;
    if (g.b1)
        g.bf ? k_gemm_tile<TM, TN, WM, WN, NS, SPLIT, true, true><<<grid, th, 0, st>>>(g)
             : k_gemm_tile<TM, TN, WM, WN, NS, SPLIT, true, false><<<grid, th, 0, st>>>(g);
    else
        g.bf ? k_gemm_tile<TM, TN, WM, WN, NS, SPLIT, false, true><<<grid, th, 0, st>>>(g)
             : k_gemm_tile<TM, TN, WM, WN, NS, SPLIT, false, false><<<grid, th, 0, st>>>(g);
    return hipGetLastError();
}

template <int TM, int TN, int WM, int WN, int NS>
hipError_t tiled(GemmArgs g, int splits, hipStream_t st)
{
    g.tiles_m = (int)cdiv(g.m, TM);
    g.tiles_n = (int)cdiv(g.n, TN);
    if (splits <= 1)
        return run_tiles<TM, TN, WM, WN, NS, false>(g, 1, st);
    const hipError_t e = run_tiles<TM, TN, WM, WN, NS, true>(g, splits, st);
    return e == hipSuccess ? join(g, splits, st) : e;
}

hipError_t launch_plan(const GemmArgs& g, int kind, int splits, hipStream_t st)
{
    switch (kind) {
    case 0: return tiled<kTileCosts[0].tm, kTileCosts[0].tn, 4, 2, 2>(g, splits, st);
    case 1: return tiled<kTileCosts[1].tm, kTileCosts[1].tn, 2, 2, 2>(g, splits, st);
    case 2: return tiled<kTileCosts[2].tm, kTileCosts[2].tn, 1, 4, 3>(g, splits, st);
    case 3: return tiled<kTileCosts[3].tm, kTileCosts[3].tn, 1, 4, 3>(g, splits, st);
    case 4: return tiled<kTileCosts[4].tm, kTileCosts[4].tn, 1, 4, 3>(g, splits, st);
    default: return few(g, st);
    }
}

}  // namespace

size_t gemm_workspace(const GemmArgs& g)
{
    if (g.k == 0)
        return 0;
    const GemmPlan p = plan_gemm(g.m, g.n, g.k, g.bf);
    return p.splits > 1 ? (size_t)p.splits * (g.m - p.main) * g.n * sizeof(float) : 0;
}

hipError_t launch_gemm(const GemmArgs& g, hipStream_t st)
{
    if (g.k == 0)
        return join(g, 0, st);
    const GemmPlan p = plan_gemm(g.m, g.n, g.k, g.bf);
    if (p.main == 0)
        return launch_plan(g, p.kind, p.splits, st);
    GemmArgs top = g, rest = g;
    top.m = p.main;
    rest.m = g.m - p.main;
    rest.a += p.main * g.k;
    rest.sa += p.main * (g.k >> 7);
    rest.c = (char*)g.c + p.main * g.n * (g.bf ? 2 : 4);
    const hipError_t e = launch_plan(top, 0, 1, st);
    return e == hipSuccess ? launch_plan(rest, p.kind, p.splits, st) : e;
}

}  // namespace fq
