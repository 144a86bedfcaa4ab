// k_swiglu.hip -- the gated activation y = silu(gate) up, silu(g) = g s(g) with
// s(g) = 1 / (1 + exp(-g)), quantized planes of its result, and its gradient
//
//   dgate = dy up s (1 + gate (1 - s)),   dup = dy gate s.
//
// Nothing crosses rows or columns but the blocks' scales, so a 128x128 tile is
// read once and leaves as rowwise and colwise planes. With e = exp(-g), s is
// 1 / (1 + e) and 1 - s is e s where the difference would cancel. The hardware's base-2
// exponential and its reciprocal are off by a unit in the last place each; the
// exponent's rounding, which would add 2^-24 |g| log2(e), and the error of its
// constant are taken back to first order, and the reciprocal refined once: s is
// off by 2.5 units at most wherever the gate lies and by 5e-8 in the mean square,
// 9e-8 without, and codes differ that much more seldom from those of the exact
// result (8192x14336: a microsecond). Where exp(-|g|) is no normal number
// it counts as zero: gates beyond 87.
//
// Bytes bound it. 8192x14336 in bf16 with both planes 8-bit: 712 MB in 138 us,
// 5.1 TB/s (a large copy reaches 5.05); its gradient 1.19 GB in 243 to 250, 4.8 TB/s.
// The scales are a word for each row and column of a tile, so that planes and
// scales of 485 MB are 533 MB of lines in the gradient. Giving each XCD an
// eighth of all tiles, in bands of 2 to 64 rows of tiles, would bring more of
// them together, but moves the times by 10% either way with the pitch of the rows (bands
// of 16: 135 and 231 us here, 94 and 157 for 8192x8192; tile_in_turn has the times of what is done).
#include <algorithm>

#include "launch.hpp"
#include "planes.hpp"

namespace fq {
namespace {

// s = 1 / (1 + exp(-g)) and 1 - s. Gates beyond what is asked for here have s = 0 or 1 - s = 0 already.
__device__ __forceinline__ void sigmoid(float g, float& s, float& rest)
{
    // log2(e) in two terms: one alone is off by 1.3e-8 of the exponent, always in one direction
    constexpr float kHi = 1.44269504f, kLo = 1.92596303e-8f;
    const float a = __builtin_amdgcn_fmed3f(g, -88.5f, 128.0f), t = a * -kHi;
    const float p = __builtin_amdgcn_exp2f(t);
    const float e = __builtin_fmaf(p, __builtin_fmaf(a, -kLo, __builtin_fmaf(a, -kHi, -t)) * 0.693147181f, p);
    const float d = 1.0f + e, r = __builtin_amdgcn_rcpf(d);
    s = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
    // The gradient's 1 + gate (1 - s) cancels around a gate of -1.28: there the difference is the one that is off by least.
    rest = g < 0.0f ? 1.0f - s : e * s;
}

// One value: y, or with BACK dgate and dup.
template <bool BACK>
__device__ __forceinline__ void gated(float gate, float up, float dy, float& first, float& second)
{
    float s, rest;
    sigmoid(gate, s, rest);
    if constexpr (BACK) {
        const float ds = dy * s;
        first = ds * up * __builtin_fmaf(gate, rest, 1.0f);
        second = ds * gate;
    } else {
        first = gate * s * up;
    }
}

// ---------------------------------------------------------------- rows alone
// Without colwise planes nothing is shared but a row's blocks: a thread takes
// eight columns of a row, and there are as many threads as that gives
// (48x18432: 3.1 us, in 128x128 tiles 5.6; the gradient of 896x7168 in blocks of 128: 10.7 and 20.4).
template <int P, bool BACK>
__global__ __launch_bounds__(kWG) void k_swiglu_rows(SwigluArgs a)
{
    const int64_t c = ((int64_t)blockIdx.x * kWG + threadIdx.x) * 8;
    const bool in = c < a.cols;
    const int64_t at = in ? c : a.cols - 8;  // past the last columns: the last ones again, not stored
    const int64_t C = BACK ? 2 * a.cols : a.cols;
    using T = PlaneTraits<P>;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        Eight gate, up, dy;
        gate.load(a.x, a.x_bf, row * a.x_stride + at);
        up.load(a.x, a.x_bf, row * a.x_stride + a.cols + at);
        if constexpr (BACK)
            dy.load(a.dy, a.dy_bf, row * a.cols + at);
        float g[8], u[8], d[8], first[8], second[8];
        gate.widen(a.x_bf, g);
        up.widen(a.x_bf, u);
        if constexpr (BACK)
            dy.widen(a.dy_bf, d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            gated<BACK>(g[e], u[e], BACK ? d[e] : 0.0f, first[e], second[e]);
        if (a.y && in) {
            store8(a.y, a.y_bf, row * C + c, first);
            if constexpr (BACK)
                store8(a.y, a.y_bf, row * C + a.cols + c, second);
        }
        if constexpr (P != kNoPlanes) {
            uint8_t* q = a.q + row * (T::kFmt == kE2M1 ? C / 2 : C);
            uint8_t* s = (uint8_t*)a.s + row * (C / T::kBlock) * (T::kMx ? 1 : 4);
            row_plane8<P>(first, c, in, q, s);
            if constexpr (BACK)
                row_plane8<P>(second, c + a.cols, in, q, s);
        }
    }
}

template <bool BACK>
hipError_t by_rows(const SwigluArgs& a, hipStream_t st)
{
    // a grid's dimension has less than 2^32 threads, and 65536 workgroups in its second
    const dim3 grid((unsigned)cdiv(a.cols, 8 * kWG), (unsigned)std::min<int64_t>(a.rows, 65535));
    switch (a.q ? a.kind : (int)kNoPlanes) {
    case kMxE4M3: k_swiglu_rows<kMxE4M3, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kMxE5M2: k_swiglu_rows<kMxE5M2, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kMxE2M1: k_swiglu_rows<kMxE2M1, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kBlockFp32: k_swiglu_rows<kBlockFp32, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kBlockPow2: k_swiglu_rows<kBlockPow2, BACK><<<grid, kWG, 0, st>>>(a); break;
    default: k_swiglu_rows<kNoPlanes, BACK><<<grid, kWG, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- tiles
// High-precision copy and planes of a tile of [R, C].
template <int P>
__device__ __forceinline__ void emit(const SwigluArgs& a, const float (&v)[8][4], TileLds& lds, const TileSpan& t,
                                     int64_t R, int64_t C)
{
    if (a.y) {
        const int c = tile_col(), r = tile_row();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c < t.cols && r + i < t.rows)
                store4v(a.y, a.y_bf, (t.r0 + r + i) * C + t.c0 + c, v[i]);
    }
    tile_planes<P>(v, lds, t, R, C, a.q, a.s, a.qt, a.st);
}

// Rows of a thread's dup that wait in LDS while dgate leaves.
constexpr int kKept = 6;

// The tile of turn t. Consecutive workgroups go to the eight XCDs in turn; a
// run of eight neighbouring tiles goes to one of them instead, whose L2 then
// has whole pieces of the rows and of their scales. The order of the whole stays
// the rows' own. (The activation and its gradient in one call, when this was
// chosen: 8192x14336 139 and 244 us, 146 and 254 without; 8192x8192 80 and 137,
// 83 and 146; runs of 2, 4, 16 and 32 in between or the same.)
__device__ __forceinline__ int64_t tile_in_turn(int64_t t, int64_t tiles)
{
    constexpr uint32_t kRun = 8;
    const uint32_t u = (uint32_t)t, first = u / (8 * kRun) * (8 * kRun);
    return first + 8 * kRun <= (uint32_t)tiles ? first + u % 8 * kRun + (u - first) / 8 : u;
}

// A 128x128 tile of gate, of up and with BACK of dy a workgroup, for colwise planes.
template <int P, bool BACK, bool XBF, bool DBF>
__global__ __launch_bounds__(kTileThreads, 4) void k_swiglu(SwigluArgs a)
{
    __shared__ __align__(16) TileLds lds;
    __shared__ u32x4 kept[BACK ? kKept : 1][kTileThreads];
    const int64_t across = cdiv(a.cols, kTileSide), tiles = across * cdiv(a.rows, kTileSide);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        int64_t tr, tc;
        tile_coords(tile_in_turn(t, tiles), across, tr, tc);
        TileSpan span = tile_span(tr, tc, a.rows, a.cols);
        const int64_t c = span.c0 + min(tile_col(), span.cols - 4);
        TileRows<XBF> gates(a.x, span, a.x_stride, c), ups(a.x, span, a.x_stride, a.cols + c);
        TileRows<DBF> dys(BACK ? a.dy : a.x, span, a.cols, c);
        float v[8][4], w[BACK ? 8 : 1][4];
        // all eight rows' loads at once; with fp32 operands of the gradient, which would not fit the registers, four's
        constexpr int kAt = BACK && !XBF ? 4 : 8;
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += kAt) {
            Four<XBF> gate[kAt], up[kAt];
            Four<DBF> dy[BACK ? kAt : 1];
#pragma unroll
            for (int i = 0; i < kAt; ++i) {
                gate[i] = gates.next();
                up[i] = ups.next();
                if constexpr (BACK)
                    dy[i] = dys.next();
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = i0; i < i0 + kAt; ++i) {
                float g[4], u[4], d[4];
                gate[i - i0].widen(g);
                up[i - i0].widen(u);
                if constexpr (BACK)
                    dy[i - i0].widen(d);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    gated<BACK>(g[e], u[e], BACK ? d[e] : 0.0f, v[i][e], w[BACK ? i : 0][e]);
                    if constexpr (BACK)
                        asm volatile("" : "+v"(w[i][e]));  // here: the compiler would keep both factors until its use
                }
                if (BACK && i < kKept) {
                    const float* d = w[BACK ? i : 0];
                    kept[i][threadIdx.x] =
                        u32x4{__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3])};
                }
                // rows one after the other: all at once would hold their intermediate values too
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (BACK) {
            emit<P>(a, v, lds, span, a.rows, 2 * a.cols);
            span.c0 += a.cols;
#pragma unroll
            for (int i = 0; i < kKept; ++i) {
                const u32x4 d = kept[i][threadIdx.x];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[i][e] = __uint_as_float(d[e]);
            }
            emit<P>(a, w, lds, span, a.rows, 2 * a.cols);
        } else {
            emit<P>(a, v, lds, span, a.rows, a.cols);
        }
    }
}

template <bool BACK, bool XBF, bool DBF>
hipError_t run(const SwigluArgs& a, hipStream_t st)
{
    const int64_t tiles = cdiv(a.rows, kTileSide) * cdiv(a.cols, kTileSide);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, 1 << 20);
    switch (a.kind) {
    case kMxE4M3: k_swiglu<kMxE4M3, BACK, XBF, DBF><<<grid, kTileThreads, 0, st>>>(a); break;
    case kMxE5M2: k_swiglu<kMxE5M2, BACK, XBF, DBF><<<grid, kTileThreads, 0, st>>>(a); break;
    case kMxE2M1: k_swiglu<kMxE2M1, BACK, XBF, DBF><<<grid, kTileThreads, 0, st>>>(a); break;
    case kBlockFp32: k_swiglu<kBlockFp32, BACK, XBF, DBF><<<grid, kTileThreads, 0, st>>>(a); break;
    default: k_swiglu<kBlockPow2, BACK, XBF, DBF><<<grid, kTileThreads, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t st)
{
    if (!a.qt)
        return a.dy ? by_rows<true>(a, st) : by_rows<false>(a, st);
    if (!a.dy)
        return a.x_bf ? run<false, true, true>(a, st) : run<false, false, true>(a, st);
    if (a.x_bf)
        return a.dy_bf ? run<true, true, true>(a, st) : run<true, true, false>(a, st);
    return a.dy_bf ? run<true, false, true>(a, st) : run<true, false, false>(a, st);
}

}  // namespace fq
