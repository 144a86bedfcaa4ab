// planes.hpp -- quantized planes of a tensor that a kernel computes: the
// recipes of k_mx.hip, k_mxfp4.hip and k_block.hip applied to fp32 values in
// registers, so that what an operator hands to the next product never lies in
// memory in high precision. The planes are those that fq_quantize makes of the
// same fp32 values, bit for bit.
#pragma once

#include "codec.hpp"
#include "launch.hpp"

namespace fq {

template <int P>
struct PlaneTraits {
    static constexpr bool kMx = P <= kMxE2M1;
    static constexpr int kFmt = P == kMxE5M2 ? (int)kE5M2 : P == kMxE2M1 ? (int)kE2M1 : (int)kE4M3;
    static constexpr int kBlock = kMx ? 32 : 128;  // elements that share a scale
};

// Multiplier of a block's values and its stored scale (an E8M0 code, or fp32 bits).
template <int P>
__device__ __forceinline__ void block_scale(float a, float& mult, uint32_t& stored)
{
    if constexpr (PlaneTraits<P>::kMx) {
        stored = mx_code<PlaneTraits<P>::kFmt>(a);
        mult = mx_multiplier(stored);
    } else if constexpr (P == kBlockPow2) {
        const uint32_t code = mx_code<kE4M3>(a);
        mult = mx_multiplier(code);
        stored = __float_as_uint(e8m0_value(code));
    } else {
        float s;
        tensor_scales(a, 448.0f, mult, s);
        stored = __float_as_uint(s);
    }
}

// ---------------------------------------------------------------- eight values of a row
__device__ __forceinline__ void load8(const void* p, bool bf, int64_t at, float* f)
{
    if (bf) {
        In<uint16_t>::unpack(ld16((const uint16_t*)p + at), f);
    } else {
        In<float>::unpack(ld16((const float*)p + at), f);
        In<float>::unpack(ld16((const float*)p + at + 4), f + 4);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
}

__device__ __forceinline__ void store8(void* p, bool bf, int64_t at, const float* f)
{
    if (bf) {
        *(u32x4*)((uint16_t*)p + at) =
            u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    } else {
        float* q = (float*)p + at;
#pragma unroll
        for (int e = 0; e < 8; e += 4)
            *(u32x4*)(q + e) = u32x4{__float_as_uint(f[e]), __float_as_uint(f[e + 1]), __float_as_uint(f[e + 2]),
                                     __float_as_uint(f[e + 3])};
    }
}

// Eight consecutive values of a row, from column c on, to the rowwise plane.
// The lanes that share a block (4 or 16, aligned) call it together; `in` is
// the same for all of them. codes and scales: the row's first.
template <int P>
__device__ __forceinline__ void row_plane8(const float* f, int64_t c, bool in, uint8_t* codes, void* scales)
{
    using T = PlaneTraits<P>;
    float mult;
    uint32_t stored;
    block_scale<P>(max_lanes<T::kBlock / 8>(absmax<8>(f)), mult, stored);
    if (!in)
        return;
    if constexpr (T::kFmt == kE2M1)
        st4_stream(codes + (c >> 1), enc8_e2m1(f, mult));
    else
        Enc8<T::kFmt, 8>::store(codes + c, f, mult);
    if ((c & (T::kBlock - 1)) == 0) {
        if constexpr (T::kMx)
            ((uint8_t*)scales)[c >> 5] = (uint8_t)stored;
        else
            ((uint32_t*)scales)[c >> 7] = stored;
    }
}

// ---------------------------------------------------------------- 128x128 tiles
// A workgroup of 256 threads holds a tile; thread t has columns 8 (t % 16) ..
// + 7 of rows 8 (t / 16) .. + 7. A row's 16 lanes read 256 contiguous bytes of
// bf16, and a wave holds 32 rows, so that an MX block of either direction lies
// within one wave.
constexpr int kTileSide = 128;

struct TileLds {
    uint8_t codes[kTileSide * 128];   // the codes of X^T
    uint32_t scale[kTileSide * 4];    // a column's amaxes, by wave, then its scales
};

// Where chunk ch (16 bytes) of column col lies. A wave writes eight bytes of
// columns 8 apart at a time and reads whole rows of eight chunks: exchanging
// odd and even columns in the upper half, and chunks by the column's group,
// leaves no bank with more than its share in either.
__device__ __forceinline__ int tile_at(int col, int ch)
{
    const int grp = col >> 3;
    return (col ^ (grp >> 3 & 1)) * 128 + ((ch ^ (grp & 7)) << 4);
}

// A tile of a [R, C] tensor: its first row and column, and how many of its 128
// rows and columns there are.
struct TileSpan {
    int64_t r0, c0;
    int rows, cols;
};

__device__ __forceinline__ TileSpan tile_span(int64_t tr, int64_t tc, int64_t R, int64_t C)
{
    const int64_t r0 = tr * kTileSide, c0 = tc * kTileSide;
    return {r0, c0, (int)min((int64_t)kTileSide, R - r0), (int)min((int64_t)kTileSide, C - c0)};
}

// Rowwise planes of a thread's 8x8 values.
template <int P>
__device__ __forceinline__ void tile_rows(const float (&v)[8][8], const TileSpan& t, int64_t C, uint8_t* q, void* s)
{
    using T = PlaneTraits<P>;
    const int c = (threadIdx.x & 15) * 8, r = (threadIdx.x >> 4) * 8;
    const int64_t pitch = T::kFmt == kE2M1 ? C / 2 : C, scales = C / T::kBlock * (T::kMx ? 1 : 4);
    uint8_t* to = q + (t.r0 + r) * pitch;
    uint8_t* to_s = (uint8_t*)s + (t.r0 + r) * scales;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        row_plane8<P>(v[i], t.c0 + c, c < t.cols && r + i < t.rows, to + i * pitch, to_s + i * scales);
}

// The maximum over the lanes 16 and 32 apart.
__device__ __forceinline__ float max_rows_of_wave(float v)
{
    const uint32_t u = __float_as_uint(v);
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(u, u, false, false));
    const uint32_t w = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(w, w, false, false));
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The colwise plane of a tile: codes of X^T [C, R], whole lines of 128 bytes.
// Values past the tile's rows are zeros. Every thread calls it; a second tile
// may follow at once.
template <int P>
__device__ __forceinline__ void tile_cols(const float (&v)[8][8], TileLds& lds, const TileSpan& t, int64_t R,
                                          uint8_t* qt, void* st)
{
    using T = PlaneTraits<P>;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        a[e] = fabsf(v[0][e]);
#pragma unroll
        for (int i = 1; i < 8; ++i)
            a[e] = fmaxf(a[e], fabsf(v[i][e]));
        a[e] = max_rows_of_wave(a[e]);
    }
    lds_barrier();  // the previous tile has been read
    if constexpr (!T::kMx) {
        if ((rg & 3) == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                lds.scale[wave * kTileSide + cg * 8 + e] = __float_as_uint(a[e]);
        lds_barrier();
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int w = 0; w < 4; ++w)
                a[e] = fmaxf(a[e], __uint_as_float(lds.scale[w * kTileSide + cg * 8 + e]));
        lds_barrier();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int col = cg * 8 + e;
        float mult;
        uint32_t stored;
        block_scale<P>(a[e], mult, stored);
        if constexpr (T::kFmt == kE2M1) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = v[i][e];
            *(uint32_t*)(lds.codes + tile_at(col, rg >> 2) + (rg & 3) * 4) = enc8_e2m1(f, mult);
        } else {
            u32x2 w;
            w[0] = enc4<T::kFmt>(v[0][e], v[1][e], v[2][e], v[3][e], mult);
            w[1] = enc4<T::kFmt>(v[4][e], v[5][e], v[6][e], v[7][e], mult);
            *(u32x2*)(lds.codes + tile_at(col, rg >> 1) + (rg & 1) * 8) = w;
        }
        if constexpr (T::kMx) {
            if ((rg & 3) == 0)
                ((uint8_t*)lds.scale)[col * 4 + wave] = (uint8_t)stored;
        } else if (rg == 0) {
            lds.scale[col] = stored;
        }
    }
    lds_barrier();
    constexpr int kChunks = T::kFmt == kE2M1 ? 4 : 8;
    const int64_t pitch = T::kFmt == kE2M1 ? R / 2 : R;
    const int bytes = T::kFmt == kE2M1 ? t.rows / 2 : t.rows;
#pragma unroll
    for (int k = 0; k < kChunks / 2; ++k) {
        const int at = k * kWG + threadIdx.x, col = at / kChunks, ch = at % kChunks;
        if (col < t.cols && ch * 16 < bytes)
            st16_stream(qt + (t.c0 + col) * pitch + (T::kFmt == kE2M1 ? t.r0 / 2 : t.r0) + ch * 16,
                        ld16(lds.codes + tile_at(col, ch)));
    }
    const int col = threadIdx.x;
    if (col < t.cols) {
        if constexpr (T::kMx) {
            uint8_t* to = (uint8_t*)st + (t.c0 + col) * (R / 32) + t.r0 / 32;
            if (t.rows == kTileSide && (R / 32 & 3) == 0)
                *(uint32_t*)to = lds.scale[col];
            else
                for (int j = 0; j < t.rows / 32; ++j)
                    to[j] = ((const uint8_t*)lds.scale)[col * 4 + j];
        } else {
            ((uint32_t*)st)[(t.c0 + col) * (R / 128) + t.r0 / 128] = lds.scale[col];
        }
    }
}

}  // namespace fq
