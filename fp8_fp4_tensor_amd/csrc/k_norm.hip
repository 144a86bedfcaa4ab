// k_norm.hip -- root-mean-square norm with the residual's addition, quantized
// planes of its result, and its gradients.
//
//   h = x + residual (rounded to h's type);  r = 1 / sqrt(mean_j h^2 + eps);  y = (h r) w
//
// With z = h r and g = dy w the gradients are
//   dh = r (g - z mean_j(g z)) + dres,   dw[j] = sum over rows of dy[j] z[j].
//
// All of it is memory traffic. A row stays in registers between its sum and
// its result, so each tensor is read and written once; only the colwise
// planes, whose blocks run over rows with different r, take a second kernel
// over 128x128 tiles that reads h again.
#include <algorithm>

#include "launch.hpp"
#include "planes.hpp"

namespace fq {
namespace {

// Sum over the wave; every lane receives it.
__device__ __forceinline__ float sum_wave(float v)
{
    v += dpp<kDppXor1>(v);
    v += dpp<kDppXor2>(v);
    v += dpp<kDppHalfMirror>(v);
    v += dpp<kDppMirror>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Sum over the TPR threads of a row. `lds` has a slot for each wave; slots of
// two calls in a row differ, so that one barrier does.
template <int TPR>
__device__ __forceinline__ float sum_row(float v, float* lds)
{
    v = sum_wave(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = v;
        lds_barrier();
        v = lds[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i)
            v += lds[i];
    }
    return v;
}

// TPR threads take a row, NV * 8 values each.
template <int TPR, int NV, int P>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm(NormArgs a)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ float sums[2][TPR < 256 ? 4 : TPR / 64];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    int64_t at[NV];
    bool in[NV];
    float w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        at[i] = (int64_t)(i * TPR + t) * 8;
        in[i] = at[i] < a.cols;
        if (in[i])
            load8(a.w, a.w_bf, at[i], w[i]);
    }
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows, turn ^= 1) {
        const int64_t row = first + sub;
        const bool live = row < a.rows;
        float f[NV][8];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (live && in[i]) {
                load8(a.x, a.x_bf, row * a.x_stride + at[i], f[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[i][e] = 0.0f;
            }
        }
        if (a.res) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!(live && in[i]))
                    continue;
                float r[8];
                load8(a.res, a.h_bf, row * a.cols + at[i], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[i][e] += r[e];
                    if (a.h_bf)
                        f[i][e] = __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[i][e]) << 16);
                }
                store8(a.h, a.h_bf, row * a.cols + at[i], f[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = __builtin_fmaf(f[i][e], f[i][e], sum);
        const float r = 1.0f / sqrtf(sum_row<TPR>(sum, sums[turn]) / (float)a.cols + a.eps);
        if (a.rstd && live && t == 0)
            a.rstd[row] = r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[i][e] = in[i] ? (f[i][e] * r) * w[i][e] : 0.0f;
            if (a.y && live && in[i])
                store8(a.y, a.y_bf, row * a.cols + at[i], f[i]);
            if constexpr (P != kNoPlanes)
                if (a.q) {
                    using T = PlaneTraits<P>;
                    row_plane8<P>(f[i], at[i], live && in[i], a.q + row * (T::kFmt == kE2M1 ? a.cols / 2 : a.cols),
                                  (uint8_t*)a.s + row * (a.cols / T::kBlock) * (T::kMx ? 1 : 4));
                }
        }
    }
}

// The colwise plane, a tile of 128 x 128 a workgroup.
template <int P, bool BF>
__global__ __launch_bounds__(kTileThreads) void k_rmsnorm_cols(NormArgs a)
{
    __shared__ __align__(16) TileLds lds;
    const int64_t across = cdiv(a.cols, kTileSide), tiles = across * cdiv(a.rows, kTileSide);
    const void* h = a.res ? a.h : a.x;
    const int64_t pitch = a.res ? a.cols : a.x_stride;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        int64_t tr, tc;
        tile_coords(t, across, tr, tc);
        const TileSpan span = tile_span(tr, tc, a.rows, a.cols);
        const int64_t c = span.c0 + min(tile_col(), span.cols - 4);
        Four<BF> raw[8];
        float r[8], w[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = span.r0 + min(tile_row() + i, span.rows - 1);
            raw[i].load(h, row * pitch + c);
            r[i] = a.rstd[row];
        }
        if (a.w_bf) {
            Four<true> b;
            b.load(a.w, c);
            b.widen(w);
        } else {
            Four<false> b;
            b.load(a.w, c);
            b.widen(w);
        }
        float v[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            raw[i].widen(v[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[i][e] = (v[i][e] * r[i]) * w[e];
        }
        tile_planes<P>(v, lds, span, a.rows, a.cols, nullptr, nullptr, a.qt, a.st);
    }
}

template <bool BF>
hipError_t cols(const NormArgs& a, hipStream_t st)
{
    const int64_t tiles = cdiv(a.rows, kTileSide) * cdiv(a.cols, kTileSide);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, 1 << 20);
    switch (a.kind) {
    case kMxE4M3: k_rmsnorm_cols<kMxE4M3, BF><<<grid, kTileThreads, 0, st>>>(a); break;
    case kMxE5M2: k_rmsnorm_cols<kMxE5M2, BF><<<grid, kTileThreads, 0, st>>>(a); break;
    case kMxE2M1: k_rmsnorm_cols<kMxE2M1, BF><<<grid, kTileThreads, 0, st>>>(a); break;
    case kBlockFp32: k_rmsnorm_cols<kBlockFp32, BF><<<grid, kTileThreads, 0, st>>>(a); break;
    default: k_rmsnorm_cols<kBlockPow2, BF><<<grid, kTileThreads, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

template <int TPR, int NV>
hipError_t rows(const NormArgs& a, hipStream_t st)
{
    constexpr int th = TPR < 256 ? 256 : TPR;
    const unsigned grid = (unsigned)std::min<int64_t>(cdiv(a.rows, th / TPR), 16384);
    switch (a.q ? a.kind : (int)kNoPlanes) {
    case kMxE4M3: k_rmsnorm<TPR, NV, kMxE4M3><<<grid, th, 0, st>>>(a); break;
    case kMxE5M2: k_rmsnorm<TPR, NV, kMxE5M2><<<grid, th, 0, st>>>(a); break;
    case kMxE2M1: k_rmsnorm<TPR, NV, kMxE2M1><<<grid, th, 0, st>>>(a); break;
    case kBlockFp32: k_rmsnorm<TPR, NV, kBlockFp32><<<grid, th, 0, st>>>(a); break;
    case kBlockPow2: k_rmsnorm<TPR, NV, kBlockPow2><<<grid, th, 0, st>>>(a); break;
    default: k_rmsnorm<TPR, NV, kNoPlanes><<<grid, th, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- gradients
// A workgroup takes every gridDim.x-th row (group of rows); what its threads
// add to dw stays in registers until its last row and leaves as one row of
// partial sums, so that the order of additions depends on the shape alone.
template <int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_backward(NormBackArgs a)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ float sums[2][TPR < 256 ? 4 : TPR / 64];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    int64_t at[NV];
    bool in[NV];
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        at[i] = (int64_t)(i * TPR + t) * 8;
        in[i] = at[i] < a.cols;
        if (in[i])
            load8(a.w, a.w_bf, at[i], w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[i][e] = 0.0f;
    }
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows, turn ^= 1) {
        const int64_t row = first + sub;
        const bool live = row < a.rows;
        const float r = live ? a.rstd[row] : 0.0f;
        float z[NV][8], g[NV][8];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool ok = live && in[i];
            if (ok) {
                load8(a.h, a.h_bf, row * a.cols + at[i], z[i]);
                load8(a.dy, a.dy_bf, row * a.cols + at[i], g[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[i][e] = ok ? z[i][e] * r : 0.0f;
                const float d = ok ? g[i][e] : 0.0f;
                dw[i][e] = __builtin_fmaf(d, z[i][e], dw[i][e]);
                g[i][e] = ok ? d * w[i][e] : 0.0f;
                dot = __builtin_fmaf(g[i][e], z[i][e], dot);
            }
        }
        const float mean = sum_row<TPR>(dot, sums[turn]) / (float)a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!(live && in[i]))
                continue;
            float d[8];
            if (a.dres) {
                load8(a.dres, a.h_bf, row * a.cols + at[i], d);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    d[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d[e] = __builtin_fmaf(r, g[i][e] - z[i][e] * mean, d[e]);
            store8(a.dx, a.h_bf, row * a.cols + at[i], d);
        }
    }
    if (a.dw) {
        float* to = a.ws + ((int64_t)blockIdx.x * kRows + sub) * a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i])
                store8(to, false, at[i], dw[i]);
    }
}

// dw = the sum of n rows of partial sums: 32 columns a workgroup, 32 rows at a
// time, each thread's rows in order and then the 32 threads of a column.
__global__ __launch_bounds__(kWG) void k_rmsnorm_dw(NormBackArgs a, int n)
{
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ f32x4 part[32][8];
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 32 + cg * 4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < a.cols)
        for (int i = rg; i < n; i += 32)
            sum += *(const f32x4*)(a.ws + (int64_t)i * a.cols + c);
    part[rg][cg] = sum;
    __syncthreads();
    if (rg > 0 || c >= a.cols)
        return;
#pragma unroll
    for (int i = 1; i < 32; ++i)
        sum += part[i][cg];
    f32x4* to = (f32x4*)(a.dw + c);
    *to = a.acc ? *to + sum : sum;
}

// Rows of partial sums (workgroups times rows at a time).
int64_t partial_rows(int64_t rows, int64_t cols)
{
    const int64_t at_once = cols <= 1024 ? 4 : 1;
    return std::min<int64_t>(cdiv(rows, at_once), 1024) * at_once;
}

template <int TPR, int NV>
hipError_t backward(const NormBackArgs& a, hipStream_t st)
{
    constexpr int th = TPR < 256 ? 256 : TPR;
    const int64_t n = partial_rows(a.rows, a.cols);
    if (n > 0)
        k_rmsnorm_backward<TPR, NV><<<(unsigned)(n / (th / TPR)), th, 0, st>>>(a);
    if (a.dw)
        k_rmsnorm_dw<<<(unsigned)cdiv(a.cols, 32), kWG, 0, st>>>(a, (int)n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st)
{
    hipError_t e = a.cols <= 512     ? rows<64, 1>(a, st)
                   : a.cols <= 1024  ? rows<64, 2>(a, st)
                   : a.cols <= 2048  ? rows<256, 1>(a, st)
                   : a.cols <= 4096  ? rows<256, 2>(a, st)
                   : a.cols <= 8192  ? rows<256, 4>(a, st)
                   : a.cols <= 16384 ? rows<512, 4>(a, st)
                                     : rows<1024, 4>(a, st);
    if (e != hipSuccess || !a.qt)
        return e;
    return (a.res ? a.h_bf : a.x_bf) ? cols<true>(a, st) : cols<false>(a, st);
}

size_t rmsnorm_workspace(int64_t rows, int64_t cols) { return (size_t)(partial_rows(rows, cols) * cols) * sizeof(float); }

hipError_t launch_rmsnorm_backward(const NormBackArgs& a, hipStream_t st)
{
    return a.cols <= 512     ? backward<64, 1>(a, st)
           : a.cols <= 1024  ? backward<64, 2>(a, st)
           : a.cols <= 2048  ? backward<256, 1>(a, st)
           : a.cols <= 4096  ? backward<256, 2>(a, st)
           : a.cols <= 8192  ? backward<256, 4>(a, st)
           : a.cols <= 16384 ? backward<512, 4>(a, st)
                             : backward<1024, 4>(a, st);
}

}  // namespace fq
