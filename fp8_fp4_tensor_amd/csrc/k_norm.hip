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
// over 128x128 tiles that reads h again. 8192x8192 in bf16 with a residual and
// both planes: 541 MB that have to move, 675 that do, in 112 us (6.0 TB/s); the gradients
// of 8192x4096 268 MB in 57 us, of which adding the weight's is 4.
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

// The columns of a thread: NV runs of eight, TPR threads apart. A thread past
// the last column repeats the row's last eight and adds nothing.
template <int TPR, int NV>
struct Columns {
    int at[NV];
    bool in[NV];
    __device__ __forceinline__ explicit Columns(int64_t cols)
    {
        const int t = threadIdx.x % TPR;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            at[i] = (i * TPR + t) * 8;
            in[i] = at[i] < cols;
            at[i] = min(at[i], (int)cols - 8);
        }
    }
};

template <int TPR, int NV>
__device__ __forceinline__ void load_weight(const void* w, bool bf, const Columns<TPR, NV>& c, float (&f)[NV][8])
{
    Eight raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        raw[i].load(w, bf, c.at[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        raw[i].widen(bf, f[i]);
}

// TPR threads take a row, NV * 8 values each. BF: x, residual and h are bf16.
template <int TPR, int NV, int P, bool BF>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm(NormArgs a)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ float sums[2][TPR < 256 ? 4 : TPR / 64];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const bool x_bf = BF || a.x_bf, h_bf = BF || a.h_bf;
    const Columns<TPR, NV> c(a.cols);
    float w[NV][8];
    load_weight(a.w, a.w_bf, c, w);
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows, turn ^= 1) {
        const bool live = first + sub < a.rows;
        const int64_t row = live ? first + sub : a.rows - 1;
        Eight x[NV], res[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            x[i].load(a.x, x_bf, row * a.x_stride + c.at[i]);
        if (a.res)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                res[i].load(a.res, h_bf, row * a.cols + c.at[i]);
        float f[NV][8];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i].widen(x_bf, f[i]);
            if (a.res) {
                float r[8];
                res[i].widen(h_bf, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[i][e] += r[e];
                    if (h_bf)
                        f[i][e] = __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[i][e]) << 16);
                }
                if (live && c.in[i])
                    store8(a.h, h_bf, row * a.cols + c.at[i], f[i]);
            }
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                part = __builtin_fmaf(f[i][e], f[i][e], part);
            sum += c.in[i] ? part : 0.0f;
        }
        const float r = 1.0f / sqrtf(sum_row<TPR>(sum, sums[turn]) / (float)a.cols + a.eps);
        if (a.rstd && live && t == 0)
            a.rstd[row] = r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[i][e] = (f[i][e] * r) * w[i][e];
            if (a.y && live && c.in[i])
                store8(a.y, a.y_bf, row * a.cols + c.at[i], f[i]);
            if constexpr (P != kNoPlanes) {
                using T = PlaneTraits<P>;
                row_plane8<P>(f[i], c.at[i], live && c.in[i], a.q + row * (T::kFmt == kE2M1 ? a.cols / 2 : a.cols),
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

template <int TPR, int NV, bool BF>
hipError_t rows(const NormArgs& a, hipStream_t st)
{
    constexpr int th = TPR < 256 ? 256 : TPR;
    const unsigned grid = (unsigned)std::min<int64_t>(cdiv(a.rows, th / TPR), 16384);
    switch (a.q ? a.kind : (int)kNoPlanes) {
    case kMxE4M3: k_rmsnorm<TPR, NV, kMxE4M3, BF><<<grid, th, 0, st>>>(a); break;
    case kMxE5M2: k_rmsnorm<TPR, NV, kMxE5M2, BF><<<grid, th, 0, st>>>(a); break;
    case kMxE2M1: k_rmsnorm<TPR, NV, kMxE2M1, BF><<<grid, th, 0, st>>>(a); break;
    case kBlockFp32: k_rmsnorm<TPR, NV, kBlockFp32, BF><<<grid, th, 0, st>>>(a); break;
    case kBlockPow2: k_rmsnorm<TPR, NV, kBlockPow2, BF><<<grid, th, 0, st>>>(a); break;
    default: k_rmsnorm<TPR, NV, kNoPlanes, BF><<<grid, th, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

// Threads of a row, so that a thread has at most 32 values and a row of up to
// 4096 columns one or two loads of each tensor.
template <bool BF>
hipError_t by_cols(const NormArgs& a, hipStream_t st)
{
    return a.cols <= 512     ? rows<64, 1, BF>(a, st)
           : a.cols <= 1024  ? rows<64, 2, BF>(a, st)
           : a.cols <= 2048  ? rows<256, 1, BF>(a, st)
           : a.cols <= 4096  ? rows<256, 2, BF>(a, st)
           : a.cols <= 8192  ? rows<256, 4, BF>(a, st)
           : a.cols <= 16384 ? rows<512, 4, BF>(a, st)
                             : rows<1024, 4, BF>(a, st);
}

// ---------------------------------------------------------------- gradients
// A workgroup takes every gridDim.x-th row (group of rows); what its threads
// add to dw stays in registers until its last row and leaves as one row of
// partial sums, so that the order of additions depends on the shape alone.
// BF: h, dy, dres and dx are bf16.
template <int TPR, int NV, bool BF>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, TPR == 512 ? 4 : 1) void k_rmsnorm_backward(NormBackArgs a)
{
    // registers for a row ahead; otherwise dres and the weight come when they are needed
    constexpr bool kAhead = TPR < 1024 || NV == 1;
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ float sums[2][TPR < 256 ? 4 : TPR / 64];
    const int sub = threadIdx.x / TPR;
    const bool h_bf = BF || a.h_bf, dy_bf = BF || a.dy_bf;
    const Columns<TPR, NV> c(a.cols);
    float w[NV][8], dw[NV][8];
    if (kAhead)
        load_weight(a.w, a.w_bf, c, w);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[i][e] = 0.0f;
    const int64_t stride = (int64_t)gridDim.x * kRows;
    Eight h[NV], dy[NV], past[NV];
    float r;
    auto load = [&](int64_t row) {
        row = min(row, a.rows - 1);
        r = a.rstd[row];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            h[i].load(a.h, h_bf, row * a.cols + c.at[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            dy[i].load(a.dy, dy_bf, row * a.cols + c.at[i]);
        if (kAhead && a.dres)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                past[i].load(a.dres, h_bf, row * a.cols + c.at[i]);
    };
    if (kAhead)
        load((int64_t)blockIdx.x * kRows + sub);
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += stride, turn ^= 1) {
        const int64_t row = first + sub;
        const bool live = row < a.rows;
        if (!kAhead)
            load(row);
        float z[NV][8], g[NV][8], d[NV][8];
        const float rstd = r;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            h[i].widen(h_bf, z[i]);
            dy[i].widen(dy_bf, g[i]);
            if (kAhead && a.dres)
                past[i].widen(h_bf, d[i]);
        }
        if (!kAhead)
            load_weight(a.w, a.w_bf, c, w);
        // The next row's values come while this one's are worked on. dx may lie over any of this row's, which are
        // here, never over the next one's before those are.
        if (kAhead)
            load(row + stride);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[i][e] *= rstd;
                if (live)
                    dw[i][e] = __builtin_fmaf(g[i][e], z[i][e], dw[i][e]);
                g[i][e] *= w[i][e];
                part = __builtin_fmaf(g[i][e], z[i][e], part);
            }
            dot += c.in[i] ? part : 0.0f;
        }
        const float mean = sum_row<TPR>(dot, sums[turn]) / (float)a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!kAhead && a.dres) {
                past[i].load(a.dres, h_bf, min(row, a.rows - 1) * a.cols + c.at[i]);
                past[i].widen(h_bf, d[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d[i][e] = __builtin_fmaf(rstd, g[i][e] - z[i][e] * mean, a.dres ? d[i][e] : 0.0f);
            if (live && c.in[i])
                store8(a.dx, h_bf, row * a.cols + c.at[i], d[i]);
        }
    }
    if (a.dw) {
        float* to = a.ws + ((int64_t)blockIdx.x * kRows + sub) * a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (c.in[i])
                store8(to, false, c.at[i], dw[i]);
    }
}

// dw = the sum of n rows of partial sums: 32 columns a workgroup, 32 rows at a
// time, each thread's rows in order and then the 32 threads of a column, as a
// tree: one after the other they would round 31 times a sum that is nearly whole.
__global__ __launch_bounds__(kWG) void k_rmsnorm_dw(NormBackArgs a, int n)
{
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ f32x4 part[32][8];
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 32 + cg * 4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < a.cols)
#pragma unroll 4
        for (int i = rg; i < n; i += 32)
            sum += *(const f32x4*)(a.ws + (int64_t)i * a.cols + c);
    part[rg][cg] = sum;
    __syncthreads();
    if (rg > 0 || c >= a.cols)
        return;
    f32x4 t[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        t[i] = part[i][cg];
#pragma unroll
    for (int half = 16; half >= 1; half /= 2)
#pragma unroll
        for (int i = 0; i < half; ++i)
            t[i] += t[i + half];
    f32x4* to = (f32x4*)(a.dw + c);
    *to = a.acc ? *to + t[0] : t[0];
}

// Workgroups of the gradient's kernel: two a CU, or one that takes four rows
// where there are fewer, for each leaves a row of partial sums that is written
// and read again (1003x7168, fp32: one row each).
int64_t back_groups(int64_t rows, int64_t at_once)
{
    const int64_t all = cdiv(rows, at_once);
    return std::min<int64_t>(all, std::max<int64_t>(256, std::min<int64_t>(512, all / 4)));
}
int64_t rows_at_once(int64_t cols) { return cols <= 1024 ? 4 : 1; }

template <int TPR, int NV, bool BF>
hipError_t backward(const NormBackArgs& a, hipStream_t st)
{
    constexpr int th = TPR < 256 ? 256 : TPR;
    const int64_t groups = back_groups(a.rows, th / TPR);
    if (groups > 0)
        k_rmsnorm_backward<TPR, NV, BF><<<(unsigned)groups, th, 0, st>>>(a);
    if (a.dw)
        k_rmsnorm_dw<<<(unsigned)cdiv(a.cols, 32), kWG, 0, st>>>(a, (int)(groups * (th / TPR)));
    return hipGetLastError();
}

template <bool BF>
hipError_t back_by_cols(const NormBackArgs& a, hipStream_t st)
{
    return a.cols <= 512     ? backward<64, 1, BF>(a, st)
           : a.cols <= 1024  ? backward<64, 2, BF>(a, st)
           : a.cols <= 2048  ? backward<256, 1, BF>(a, st)
           : a.cols <= 4096  ? backward<512, 1, BF>(a, st)
           : a.cols <= 8192  ? backward<1024, 1, BF>(a, st)
           : a.cols <= 16384 ? backward<1024, 2, BF>(a, st)
                             : backward<1024, 4, BF>(a, st);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st)
{
    const hipError_t e = a.x_bf && (a.h_bf || !a.res) ? by_cols<true>(a, st) : by_cols<false>(a, st);
    if (e != hipSuccess || !a.qt)
        return e;
    return (a.res ? a.h_bf : a.x_bf) ? cols<true>(a, st) : cols<false>(a, st);
}

size_t rmsnorm_workspace(int64_t rows, int64_t cols)
{
    const int64_t n = rows_at_once(cols);
    return (size_t)(back_groups(rows, n) * n * cols) * sizeof(float);
}

hipError_t launch_rmsnorm_backward(const NormBackArgs& a, hipStream_t st)
{
    return a.h_bf && a.dy_bf ? back_by_cols<true>(a, st) : back_by_cols<false>(a, st);
}

}  // namespace fq
