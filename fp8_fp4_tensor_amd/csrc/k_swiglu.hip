// k_swiglu.hip -- the gated activation y = silu(gate) up, silu(g) = g s(g) with
// s(g) = 1 / (1 + exp(-g)), quantized planes of its result, and its gradient
//
//   dgate = dy up s (1 + gate (1 - s)),   dup = dy gate s.
//
// Nothing crosses rows or columns but the blocks' scales, so a 128x128 tile is
// read once and leaves as rowwise and colwise planes. The exponential is that
// of -|g| in base 2, which neither overflows nor cancels: with e = exp(-|g|)
// and q = 1 / (1 + e), s and 1 - s are q and e q, the larger one for the sign
// of g that has it. The hardware's base-2 exponential and reciprocal are off
// by a unit in the last place each, the exponent's own rounding by 2^-24 |g|
// log2(e): together below 2^-18 for |g| < 40. Below -87, exp(-|g|) is no
// normal number and counts as zero.
#include <algorithm>

#include "launch.hpp"
#include "planes.hpp"

namespace fq {
namespace {

// s = 1 / (1 + exp(-g)) and 1 - s
__device__ __forceinline__ void sigmoid(float g, float& s, float& rest)
{
    const float e = __builtin_amdgcn_exp2f(fabsf(g) * -1.44269504f);
    const float q = __builtin_amdgcn_rcpf(1.0f + e), u = e * q;
    s = g < 0.0f ? u : q;
    rest = g < 0.0f ? q : u;
}

// Planes and high-precision copy of a thread's 8x8 results, a tile of [R, C].
template <int P>
__device__ __forceinline__ void emit(const SwigluArgs& a, const float (&v)[8][8], TileLds& lds, const TileSpan& t,
                                     int64_t R, int64_t C)
{
    if (a.y) {
        const int c = (threadIdx.x & 15) * 8, r = (threadIdx.x >> 4) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c < t.cols && r + i < t.rows)
                store8(a.y, a.y_bf, (t.r0 + r + i) * C + t.c0 + c, v[i]);
    }
    if constexpr (P != kNoPlanes) {
        if (a.q)
            tile_rows<P>(v, t, C, a.q, a.s);
        if (a.qt)
            tile_cols<P>(v, lds, t, R, a.qt, a.st);
    }
}

template <int P, bool BACK>
__global__ __launch_bounds__(kWG) void k_swiglu(SwigluArgs a)
{
    __shared__ __align__(16) TileLds lds;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t across = cdiv(a.cols, kTileSide), tiles = across * cdiv(a.rows, kTileSide);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        int64_t tr, tc;
        tile_coords(t, across, tr, tc);
        TileSpan span = tile_span(tr, tc, a.rows, a.cols);
        const int64_t r = span.r0 + rg * 8, c = span.c0 + cg * 8;
        float v[8][8], u[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool ok = cg * 8 < span.cols && rg * 8 + i < span.rows;
            if (ok) {
                load8(a.x, a.x_bf, (r + i) * a.x_stride + c, v[i]);
                load8(a.x, a.x_bf, (r + i) * a.x_stride + a.cols + c, u[i]);
            }
            float d[8];
            if constexpr (BACK)
                if (ok)
                    load8(a.dy, a.dy_bf, (r + i) * a.cols + c, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gate = ok ? v[i][e] : 0.0f, up = ok ? u[i][e] : 0.0f;
                float s, rest;
                sigmoid(gate, s, rest);
                if constexpr (BACK) {
                    const float dy = ok ? d[e] : 0.0f, ds = dy * s;
                    v[i][e] = ds * up * __builtin_fmaf(gate, rest, 1.0f);
                    u[i][e] = ds * gate;
                } else {
                    v[i][e] = gate * s * up;
                }
            }
        }
        if constexpr (BACK) {
            emit<P>(a, v, lds, span, a.rows, 2 * a.cols);
            span.c0 += a.cols;
            emit<P>(a, u, lds, span, a.rows, 2 * a.cols);
        } else {
            emit<P>(a, v, lds, span, a.rows, a.cols);
        }
    }
}

template <bool BACK>
hipError_t run(const SwigluArgs& a, hipStream_t st)
{
    const int64_t tiles = cdiv(a.rows, kTileSide) * cdiv(a.cols, kTileSide);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, 1 << 20);
    switch (a.q || a.qt ? a.kind : (int)kNoPlanes) {
    case kMxE4M3: k_swiglu<kMxE4M3, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kMxE5M2: k_swiglu<kMxE5M2, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kMxE2M1: k_swiglu<kMxE2M1, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kBlockFp32: k_swiglu<kBlockFp32, BACK><<<grid, kWG, 0, st>>>(a); break;
    case kBlockPow2: k_swiglu<kBlockPow2, BACK><<<grid, kWG, 0, st>>>(a); break;
    default: k_swiglu<kNoPlanes, BACK><<<grid, kWG, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t st) { return a.dy ? run<true>(a, st) : run<false>(a, st); }

}  // namespace fq
