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

// Few rows of A (m <= 16 * MT): one workgroup computes 16 * NT columns; its
// waves take the blocks of k in turn and their sums meet in LDS, in wave
// order. Nothing is reused but A (from L2), so operands go straight from
// memory to the matrix unit's registers.
template <int MT, int NT, int NW, bool B1, bool BF>
__global__ __launch_bounds__(NW * 64) void k_gemm_few(GemmArgs g)
{
    __shared__ f32x4 part[NW][MT * NT][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = lane & 15, grp = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int nb = (int)(g.k >> 7);
    const uint8_t *pa[MT], *pb[NT];
    const float *psa[MT], *psb[NT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t i = min(m0 + t * 16 + row, g.m - 1);  // rows past m repeat the last one and are not stored
        pa[t] = g.a + i * g.k + grp * 16;
        psa[t] = g.sa + i * nb;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t j = min(n0 + t * 16 + row, g.n - 1);
        pb[t] = g.b + j * g.k + grp * 16;
        psb[t] = B1 ? nullptr : g.sb + (min(n0 + t * 16, g.n - 1) >> 7) * nb;
    }
    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
            acc[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = w; b < nb; b += NW) {
        i32x8 fa[MT], fb[NT];
        float s[MT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            fb[t] = join(ld16_stream(pb[t] + (int64_t)b * 128), ld16_stream(pb[t] + (int64_t)b * 128 + 64));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            fa[t] = join(ld16(pa[t] + (int64_t)b * 128), ld16(pa[t] + (int64_t)b * 128 + 64));
            s[t] = psa[t][b];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (B1) {
                float sb[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sb[e] = g.sb[min(n0 + t * 16 + grp * 4 + e, g.n - 1) * nb + b];
#pragma unroll
                for (int u = 0; u < MT; ++u) {
                    const f32x4 p = mfma_block<BF>(fb[t], fa[u]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[t][u][e] = __builtin_fmaf(p[e], s[u] * sb[e], acc[t][u][e]);
                }
            } else {
                const float sb = psb[t][b];
#pragma unroll
                for (int u = 0; u < MT; ++u) {
                    const f32x4 p = mfma_block<BF>(fb[t], fa[u]);
                    const float c = s[u] * sb;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[t][u][e] = __builtin_fmaf(p[e], c, acc[t][u][e]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
            part[w][t * MT + u][lane] = acc[t][u];
    __syncthreads();
    for (int q = w; q < MT * NT; q += NW) {
        f32x4 v = part[0][q][lane];
#pragma unroll
        for (int x = 1; x < NW; ++x)
            v += part[x][q][lane];
        const int t = q / MT, u = q - t * MT;
        const int64_t i = m0 + u * 16 + row;
        if (i < g.m)
            store4<BF>(g.c, i, n0 + t * 16 + grp * 4, g.n, v, g.acc);
    }
}

template <int MT, int NT, int NW>
hipError_t few(const GemmArgs& g, hipStream_t st)
{
    const dim3 grid((unsigned)cdiv(g.n, 16 * NT), (unsigned)cdiv(g.m, 16 * MT));
    if (g.b1)
        g.bf ? k_gemm_few<MT, NT, NW, true, true><<<grid, NW * 64, 0, st>>>(g)
             : k_gemm_few<MT, NT, NW, true, false><<<grid, NW * 64, 0, st>>>(g);
    else
        g.bf ? k_gemm_few<MT, NT, NW, false, true><<<grid, NW * 64, 0, st>>>(g)
             : k_gemm_few<MT, NT, NW, false, false><<<grid, NW * 64, 0, st>>>(g);
    return hipGetLastError();
}

// ---------------------------------------------------------------- many rows
// One workgroup computes a TM x TN tile of C, WM x WN waves of
// (TM/WM) x (TN/WN). A step is one scale block: TM + TN rows of 128 bytes
// come straight from memory into LDS (16 bytes a lane, no registers), one
// step ahead of the products. The 16-byte chunk c of row r is kept at chunk
// c ^ (r % 8) of its row, so that eight lanes reading one chunk of eight rows
// meet no bank twice; the transfer writes LDS in lane order, so it is the
// lane's source address that carries the permutation.

// 64 lanes' 16 (or 4) bytes each -> LDS at `to`, in lane order. Written as
// assembly because the compiler, which cannot tell the two stages apart,
// would wait for every transfer before the next read of LDS; there is no
// output register, and the waits are those of the step loop. M0 holds the
// LDS address and needs one wait state before its use; nothing else here uses
// it.
template <int BYTES>
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, uint32_t to, int lane_offset, int offset)
{
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :
                     : "s"(to), "v"(lane_offset), "s"(r), "s"(offset)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                     :
                     : "s"(to), "v"(lane_offset), "s"(r), "s"(offset)
                     : "memory");
}

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

template <int TM, int TN, int WM, int WN, bool B1, bool BF>
struct Tile {
    static constexpr int kNW = WM * WN;
    static constexpr int kMT = TM / WM / 16, kNT = TN / WN / 16;
    static_assert(B1 || TN / WN <= 128, "a wave's columns share a 128x128 scale");
    struct alignas(1024) Stage {
        uint8_t a[TM * 128], b[TN * 128];
        float sa[TM], sb[B1 ? TN : 64];
    };
};

template <int TM, int TN, int WM, int WN, bool B1, bool BF>
__global__ __launch_bounds__(WM* WN * 64) void k_gemm_tile(GemmArgs g)
{
    using T = Tile<TM, TN, WM, WN, B1, BF>;
    constexpr int NW = T::kNW, MT = T::kMT, NT = T::kNT;
    constexpr int IA = TM / 8 / NW, IB = TN / 8 / NW;  // transfers of 8 rows a wave issues
    static_assert(TM % (8 * NW) == 0 && TN % (8 * NW) == 0, "whole transfers");
    __shared__ typename T::Stage stage[2];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, grp = lane >> 4;
    int64_t tm, tn;
    tile_of(g, tm, tn);
    const int64_t m0 = tm * TM, n0 = tn * TN;
    const int nb = (int)(g.k >> 7);
    const int rows_a = (int)min((int64_t)TM, g.m - m0), rows_b = (int)min((int64_t)TN, g.n - n0);
    const uint8_t* pa = g.a + m0 * g.k;
    const uint8_t* pb = g.b + n0 * g.k;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)pa, 0, (int)(rows_a * g.k), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)pb, 0, (int)(rows_b * g.k), 0x00020000);
    const __amdgpu_buffer_rsrc_t rsa =
        __builtin_amdgcn_make_buffer_rsrc((void*)(g.sa + m0 * nb), 0, rows_a * nb * 4, 0x00020000);
    const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(g.sb + (B1 ? n0 : n0 >> 7) * nb), 0, (B1 ? rows_b : (rows_b + 127) >> 7) * nb * 4, 0x00020000);
    // rows past the last repeat it, so every source address is inside; they are not stored
    int va[IA], vb[IB], vsa, vsb;
    const int sub = lane >> 3, chunk = (lane & 7) ^ sub;
#pragma unroll
    for (int i = 0; i < IA; ++i)
        va[i] = min((w * IA + i) * 8 + sub, rows_a - 1) * (int)g.k + chunk * 16;
#pragma unroll
    for (int i = 0; i < IB; ++i)
        vb[i] = min((w * IB + i) * 8 + sub, rows_b - 1) * (int)g.k + chunk * 16;
    vsa = min(w * 64 + lane, rows_a - 1) * nb * 4;
    vsb = min((w - TM / 64) * 64 + lane, (B1 ? rows_b : (rows_b + 127) >> 7) - 1) * nb * 4;

    const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)stage;
    auto fill = [&](int which, int b) {
        const uint32_t to = at + which * (uint32_t)sizeof(typename T::Stage);
#pragma unroll
        for (int i = 0; i < IB; ++i)
            to_lds<16>(rb, to + offsetof(typename T::Stage, b) + (w * IB + i) * 1024, vb[i], b * 128);
#pragma unroll
        for (int i = 0; i < IA; ++i)
            to_lds<16>(ra, to + (w * IA + i) * 1024, va[i], b * 128);
        if (w < TM / 64)
            to_lds<4>(rsa, to + offsetof(typename T::Stage, sa) + w * 256, vsa, b * 4);
        else if (w < TM / 64 + (B1 ? TN / 64 : 1))
            to_lds<4>(rsb, to + offsetof(typename T::Stage, sb) + (w - TM / 64) * 256, vsb, b * 4);
    };
    const int wm = w / WN, wn = w % WN;
    const int c0 = ((grp ^ (row & 7)) * 16), c1 = c0 ^ 64;
    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
            acc[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto work = [&](const typename T::Stage& s) {
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
        // the next column tile's operand is read during this one's products;
        // the fences keep the scheduler from reading them all at once, which
        // would not fit the registers
        i32x8 fb = join(ld16(qb + c0), ld16(qb + c1));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            i32x8 next = fb;
            if (t + 1 < NT)
                next = join(ld16(qb + (t + 1) * 2048 + c0), ld16(qb + (t + 1) * 2048 + c1));
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
            fb = next;
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Each wave waits for its own transfers before the barrier; after it the
    // step's stage is whole, and every wave has read the other one.
    fill(0, 0);
    for (int b = 0; b < nb; ++b) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (b + 1 < nb)
            fill((b + 1) & 1, b + 1);
        work(stage[b & 1]);
    }
#pragma unroll
    for (int u = 0; u < MT; ++u) {
        const int64_t i = m0 + wm * (TM / WM) + u * 16 + row;
        if (i < g.m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                store4<BF>(g.c, i, n0 + wn * (TN / WN) + t * 16 + grp * 4, g.n, acc[t][u], g.acc);
    }
}

template <int TM, int TN, int WM, int WN>
hipError_t tiled(GemmArgs g, hipStream_t st)
{
    g.tiles_m = (int)cdiv(g.m, TM);
    g.tiles_n = (int)cdiv(g.n, TN);
    const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n));
    constexpr int th = WM * WN * 64;
    if (g.b1)
        g.bf ? k_gemm_tile<TM, TN, WM, WN, true, true><<<grid, th, 0, st>>>(g)
             : k_gemm_tile<TM, TN, WM, WN, true, false><<<grid, th, 0, st>>>(g);
    else
        g.bf ? k_gemm_tile<TM, TN, WM, WN, false, true><<<grid, th, 0, st>>>(g)
             : k_gemm_tile<TM, TN, WM, WN, false, false><<<grid, th, 0, st>>>(g);
    return hipGetLastError();
}

}  // namespace

size_t gemm_workspace(const GemmArgs&) { return 0; }

hipError_t launch_gemm(const GemmArgs& g, hipStream_t st)
{
    if (g.m <= 16 || g.k == 0)
        return few<1, 1, 8>(g, st);
    if (g.m <= 64)
        return few<4, 2, 4>(g, st);
    if (cdiv(g.m, 256) * cdiv(g.n, 256) >= 256)
        return tiled<256, 256, 4, 2>(g, st);
    return tiled<128, 128, 2, 2>(g, st);
}

}  // namespace fq
