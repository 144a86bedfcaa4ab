// planes.hpp -- quantized planes of a tensor that a kernel computes: the
// recipes of k_mx.hip, k_mxfp4.hip and k_block.hip applied to fp32 values in
// registers, so that what an operator hands to the next product never lies in
// memory in high precision. The planes are those that fq_quantize makes of the
// same fp32 values, bit for bit.
#pragma once

#include <type_traits>

#include "codec.hpp"
#include "launch.hpp"
#include "plan.hpp"

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
// As loaded, and widened. A kernel whose types are a call's own loads all its
// values before it widens the first: either is a branch that all lanes take
// alike, but a load and its use within one branch would wait for each other.
struct Eight {
    u32x4 lo, hi;  // bf16: lo alone
    __device__ __forceinline__ void load(const void* p, bool bf, int64_t at)
    {
        if (bf) {
            lo = ld16((const uint16_t*)p + at);
        } else {
            lo = ld16((const float*)p + at);
            hi = ld16((const float*)p + at + 4);
        }
    }
    __device__ __forceinline__ void widen(bool bf, float* f) const
    {
        if (bf) {
            In<uint16_t>::unpack(lo, f);
        } else {
            In<float>::unpack(lo, f);
            In<float>::unpack(hi, f + 4);
        }
    }
};

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
// A workgroup of 512 threads holds a tile; thread t has columns 4 (t % 32) ..
// + 3 of rows 8 (t / 32) .. + 7: a row's 32 lanes read 256 contiguous bytes of
// bf16, eight of them have an MX block of the row, and 32 values a thread leave
// room for four waves a SIMD (64 values, two columns more of lanes, left two,
// and the gated activation's gradient one: 623 us for 8192x14336).
constexpr int kTileSide = 128;
constexpr int kTileThreads = 512;

struct TileLds {
    uint8_t codes[kTileSide * 128];     // the codes of X^T
    uint32_t amax[8][kTileSide];        // of a wave's 16 rows
    uint32_t scale[kTileSide];          // a column's scales: four E8M0 codes, or one fp32
    uint32_t row_scale[kTileSide];      // a row's
    float row_mult[kTileThreads / 8][8];  // multipliers of eight rows' MX blocks
};

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

// This thread's first column and row in a tile.
__device__ __forceinline__ int tile_col() { return (threadIdx.x & 31) * 4; }
__device__ __forceinline__ int tile_row() { return (threadIdx.x >> 5) * 8; }

// Four consecutive values, as loaded and widened. Loads come first and all at
// once; a row or column past the tile's last repeats it, so every address is
// inside, and its values are not stored: blocks are whole or absent.
template <bool BF>
struct Four {
    typename std::conditional<BF, u32x2, u32x4>::type raw;
    __device__ __forceinline__ void load(const void* p, int64_t at)
    {
        if constexpr (BF)
            raw = __builtin_nontemporal_load((const u32x2*)((const uint16_t*)p + at));
        else
            raw = __builtin_nontemporal_load((const u32x4*)((const float*)p + at));
    }
    __device__ __forceinline__ void widen(float* f) const
    {
        if constexpr (BF) {
            f[0] = bf16_lo(raw[0]);
            f[1] = bf16_hi(raw[0]);
            f[2] = bf16_lo(raw[1]);
            f[3] = bf16_hi(raw[1]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = __uint_as_float(raw[e]);
        }
    }
};

// A thread's rows of a tile, one behind the other: a pointer that moves on by a
// row, and stays at the tile's last. (Eight addresses at once would hold 16
// registers for each tensor.)
template <bool BF>
struct TileRows {
    const char* p;
    int64_t step;
    int left;  // rows behind this one
    __device__ __forceinline__ TileRows(const void* base, const TileSpan& t, int64_t pitch, int64_t col)
    {
        constexpr int kBytes = BF ? 2 : 4;
        const int r = min(tile_row(), t.rows - 1);
        p = (const char*)base + ((t.r0 + r) * pitch + col) * kBytes;
        step = pitch * kBytes;
        left = t.rows - 1 - r;
    }
    __device__ __forceinline__ Four<BF> next()
    {
        Four<BF> f;
        f.load(p, 0);
        p += left > 0 ? step : 0;
        --left;
        return f;
    }
};

__device__ __forceinline__ void store4v(void* p, bool bf, int64_t at, const float* f)
{
    if (bf)
        *(u32x2*)((uint16_t*)p + at) = u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
    else
        *(u32x4*)((float*)p + at) =
            u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
}

// Where chunk ch (16 bytes) of column col lies. A wave writes 16 bytes of
// columns 4 apart at a time (two lanes, 8 rows each) and reads whole rows of
// eight chunks: exchanging odd and even columns in every other eight of them,
// and chunks by the column's group, leaves no bank with more than its share in
// either.
__device__ __forceinline__ int tile_at(int col, int ch)
{
    const int grp = col >> 2;
    return (col ^ (grp >> 3 & 1)) * 128 + ((ch ^ (grp & 7)) << 4);
}

// The scales of eight lanes' MX blocks, eight rows each: exchanging halves, each
// lane comes to the largest magnitude of one row's block: seven exchanges,
// where all lanes knowing all eight takes 24 and computes each scale eight
// times (the gated activation of 8192x14336: 136 us for 141). The multipliers go
// round through LDS within the wave, the codes to the tile's.
template <int P>
__device__ __forceinline__ void row_scales(const float (&v)[8][4], TileLds& lds, float (&mult)[8])
{
    const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2, b2 = threadIdx.x & 4;
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m[i] = absmax<4>(v[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m[i] = fmaxf(b2 ? m[i + 4] : m[i], dpp<kDppHalfMirror>(b2 ? m[i] : m[i + 4]));
#pragma unroll
    for (int i = 0; i < 2; ++i)
        m[i] = fmaxf(b0 ? m[i + 2] : m[i], dpp<kDppXor1>(b0 ? m[i] : m[i + 2]));
    float own;
    uint32_t stored;
    block_scale<P>(fmaxf(b1 ? m[1] : m[0], dpp<kDppXor2>(b1 ? m[0] : m[1])), own, stored);
    const int row = 4 * b2 + 2 * b0 + b1;
    lds.row_mult[threadIdx.x >> 3][row] = own;
    ((uint8_t*)lds.row_scale)[(tile_row() + row) * 4 + (tile_col() >> 5)] = (uint8_t)stored;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
#pragma unroll
    for (int i = 0; i < 8; ++i)
        mult[i] = lds.row_mult[threadIdx.x >> 3][i];
}

// A tile's scales of one row of a plane with `per` scales a row: `codes` E8M0
// codes, or one fp32, from scale `first` on.
template <bool MX>
__device__ __forceinline__ void store_scales(void* plane, int64_t row, int64_t per, int64_t first, int codes, uint32_t word)
{
    const int64_t at = row * per + first;
    if constexpr (!MX) {
        ((uint32_t*)plane)[at] = word;
    } else {
        uint8_t* to = (uint8_t*)plane + at;
        switch (scale_store_bytes(per, first, codes)) {
        case 4: *(uint32_t*)to = word; break;
        case 2:
            ((uint16_t*)to)[0] = (uint16_t)word;
            ((uint16_t*)to)[1] = (uint16_t)(word >> 16);
            break;
        default:
            for (int j = 0; j < codes; ++j)
                to[j] = (uint8_t)(word >> 8 * j);
        }
    }
}

// Planes of a tile's values: the rowwise one if q, the colwise one (codes of
// X^T [C, R], whole lines of 128 bytes) if qt. Every thread calls it; a second
// tile may follow at once.
template <int P>
__device__ __forceinline__ void tile_planes(const float (&v)[8][4], TileLds& lds, const TileSpan& t, int64_t R, int64_t C,
                                            uint8_t* q, void* s, uint8_t* qt, void* st)
{
    using T = PlaneTraits<P>;
    constexpr bool kPacked = T::kFmt == kE2M1;
    const int c = tile_col(), r = tile_row(), wave = threadIdx.x >> 6;
    float a[4];
    if (qt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = fabsf(v[0][e]);
#pragma unroll
            for (int i = 1; i < 8; ++i)
                a[e] = fmaxf(a[e], fabsf(v[i][e]));
            // the wave's other eight rows
            const uint32_t u = __float_as_uint(a[e]);
            const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
            a[e] = fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
        }
    }
    lds_barrier();  // the previous tile has been read
    if (qt && (threadIdx.x & 32) == 0)
        *(u32x4*)&lds.amax[wave][c] =
            u32x4{__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3])};
    if (q) {
        const int64_t pitch = kPacked ? C / 2 : C;
        uint8_t* to = q + (t.r0 + r) * pitch + (kPacked ? (t.c0 + c) / 2 : t.c0 + c);
        const bool in = c < t.cols;
        float mults[8];
        if constexpr (T::kMx)
            row_scales<P>(v, lds, mults);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float mult;
            if constexpr (T::kMx) {
                mult = mults[i];
            } else {
                uint32_t stored;
                block_scale<P>(max_lanes<T::kBlock / 4>(absmax<4>(v[i])), mult, stored);
                if ((threadIdx.x & 31) == 0)
                    lds.row_scale[r + i] = stored;
            }
            if constexpr (kPacked) {
                // two lanes' nibbles leave as one word
                const float f[8] = {v[i][0], v[i][1], v[i][2], v[i][3], 0.0f, 0.0f, 0.0f, 0.0f};
                const uint32_t half = enc8_e2m1(f, mult) & 0xFFFFu;
                const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)half, kDppXor1, 0xF, 0xF, false);
                if (in && r + i < t.rows && (threadIdx.x & 1) == 0)
                    st4_stream(to + i * pitch, half | other << 16);
            } else if (in && r + i < t.rows) {
                st4_stream(to + i * pitch, enc4<T::kFmt>(v[i][0], v[i][1], v[i][2], v[i][3], mult));
            }
        }
    }
    lds_barrier();
    if (q && threadIdx.x < t.rows) {
        const int64_t per = C / T::kBlock, first = t.c0 / T::kBlock;
        store_scales<T::kMx>(s, t.r0 + threadIdx.x, per, first, t.cols / 32, lds.row_scale[threadIdx.x]);
    }
    if (!qt)
        return;
    // the rows of a column's block: those of two waves, or of all
    u32x4 m[T::kMx ? 2 : 8];
#pragma unroll
    for (int w = 0; w < (T::kMx ? 2 : 8); ++w)
        m[w] = *(const u32x4*)&lds.amax[T::kMx ? (wave & ~1) + w : w][c];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float all = __uint_as_float(m[0][e]);
#pragma unroll
        for (int w = 1; w < (T::kMx ? 2 : 8); ++w)
            all = fmaxf(all, __uint_as_float(m[w][e]));
        float mult;
        uint32_t stored;
        block_scale<P>(all, mult, stored);
        const int col = c + e;
        if constexpr (kPacked) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = v[i][e];
            *(uint32_t*)(lds.codes + tile_at(col, r >> 5) + (r >> 1 & 15)) = enc8_e2m1(f, mult);
        } else {
            u32x2 w;
            w[0] = enc4<T::kFmt>(v[0][e], v[1][e], v[2][e], v[3][e], mult);
            w[1] = enc4<T::kFmt>(v[4][e], v[5][e], v[6][e], v[7][e], mult);
            *(u32x2*)(lds.codes + tile_at(col, r >> 4) + (r & 8)) = w;
        }
        if constexpr (T::kMx) {
            if ((r & 31) == 0)
                ((uint8_t*)lds.scale)[col * 4 + (r >> 5)] = (uint8_t)stored;
        } else if (r == 0) {
            lds.scale[col] = stored;
        }
    }
    lds_barrier();
    constexpr int kChunks = kPacked ? 4 : 8;
    const int64_t pitch = kPacked ? R / 2 : R;
    const int bytes = kPacked ? t.rows / 2 : t.rows;
#pragma unroll
    for (int k = 0; k < kChunks * kTileSide / kTileThreads; ++k) {
        const int at = k * kTileThreads + threadIdx.x, col = at / kChunks, ch = at % kChunks;
        if (col < t.cols && ch * 16 < bytes)
            st16_stream(qt + (t.c0 + col) * pitch + (kPacked ? t.r0 / 2 : t.r0) + ch * 16, ld16(lds.codes + tile_at(col, ch)));
    }
    if (threadIdx.x < t.cols) {
        const int64_t per = R / T::kBlock, first = t.r0 / T::kBlock;
        store_scales<T::kMx>(st, t.c0 + threadIdx.x, per, first, t.rows / 32, lds.scale[threadIdx.x]);
    }
}

}  // namespace fq
