// mx_operand.hpp -- how the matrix instructions of gfx950 take MX operands.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over 128
// elements, each side of its own 8- or 4-bit type, and scales every run of 32
// elements of a row by its E8M0 code. Lane l holds part of row l % 16; with
// g = l / 16 it supplies the 16-byte chunks g and 4 + g of the row's 128 bytes
// (8-bit elements) or chunk g of its 64 bytes (4-bit), and in its lowest byte
// the scale of block g, wherever that block's elements are. The accumulator
// enters the sum in fp32.
//
// Its sums. Products of two 4-bit values add up exactly within a block, and
// with 1e-7 relative error over 14336 elements whose blocks span 12 binades.
// With an 8-bit side the instruction aligns the products before it adds them
// and keeps few bits below the largest: 1.5e-5 of the result in the mean
// square for two 8-bit sides, 1.7e-6 for one, however long the sum. Beside
// the rounding of a bf16 result (1.7e-3) that is nothing; an fp32 result with
// an 8-bit side takes its operands widened to bf16 instead, scale included
// (exact), and v_mfma_f32_16x16x32_bf16, which is off by 1e-7, at half the rate.
#pragma once

#include "codec.hpp"
#include "matrix.hpp"

namespace fq {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// the instruction's number for an element type
template <int F>
constexpr int kMfmaType = F == kE4M3 ? 0 : F == kE5M2 ? 1 : 4;

// bytes of n elements
template <int F>
__host__ __device__ constexpr int64_t mx_bytes(int64_t n)
{
    return F == kE2M1 ? n >> 1 : n;
}

// Whether results of this kind take widened operands.
template <int FA, int FB, bool F32>
constexpr bool kWidened = F32 && !(FA == kE2M1 && FB == kE2M1);

template <int FR, int FC>
__device__ __forceinline__ f32x4 mfma_mx(i32x8 rows, uint32_t rows_scale, i32x8 cols, uint32_t cols_scale, f32x4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(rows, cols, c, kMfmaType<FR>, kMfmaType<FC>, 0,
                                                            (int)rows_scale, 0, (int)cols_scale);
}

// Elements 8e .. 8e+7 of a lane's 32, as bf16 times the block's scale.
template <int F>
__device__ __forceinline__ bf16x8 widen8(i32x8 v, int e, float scale)
{
    bf16x2 r[4];
    if constexpr (F == kE2M1) {
        const uint32_t w = (uint32_t)v[e];
        r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
        r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
        r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
        r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = (uint32_t)v[2 * e + h];
            if constexpr (F == kE4M3) {
                r[2 * h] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
                r[2 * h + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
            } else {
                r[2 * h] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, false);
                r[2 * h + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, true);
            }
        }
    }
    return bf16x8{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

// ---------------------------------------------------------------- beyond fp32's range
// A widened value is code times scale, which a scale near the top of E8M0's
// range takes past fp32's largest, to infinity, though the product with a
// small value of the other side is moderate (448 * 2^123 times 2^-107). An
// infinite operand leaves no finite sum, so sums that are finite are right as
// they are. Each wave adds up the others again where a row's scales can be the
// cause, a block at a time: 32 products of unscaled codes, which are exact in
// bf16, and their sum times both scales. Data without such scales pays for a
// look at its sums, and a few us a tile where they are infinite or NaN for another reason.

// The largest scale code that keeps every element finite: 1.75 * 2^(8 + 119), 1.75 * 2^(15 + 112), 1.5 * 2^(2 + 125).
template <int F>
constexpr int kTopScale = F == kE4M3 ? 246 : F == kE5M2 ? 239 : 252;

// Whether one of a row's scales [from, to) is larger (255 is no number, whatever it meets); lanes grp = 0, 1 .. of a row
// look at a part each.
template <int F, int S>
__device__ __forceinline__ bool past_top(const uint8_t* scales, int64_t from, int64_t to, int grp)
{
    int top = 0;
#pragma unroll 8
    for (int64_t b = from + grp; b < to; b += 64 / S) {
        const int c = scales[b];
        top = c == 255 ? top : max(top, c);
    }
#pragma unroll
    for (int x = S; x < 64; x *= 2)
        top = max(top, __shfl_xor(top, x));
    return top > kTopScale<F>;
}

// Elements 8p .. 8p+7 of a row's block b, unscaled.
template <int F>
__device__ __forceinline__ bf16x8 block8(const uint8_t* row, int64_t b, int p)
{
    i32x8 v{};
    if constexpr (F == kE2M1) {
        v[0] = *(const int*)(row + b * 16 + p * 4);
    } else {
        const u32x2 w = *(const u32x2*)(row + b * 32 + p * 8);
        v[0] = (int)w[0];
        v[1] = (int)w[1];
    }
    return widen8<F>(v, 0, 1.0f);
}

template <int S>
struct MxAcc;
template <>
struct MxAcc<16> {
    typedef f32x4 T;
};
template <>
struct MxAcc<32> {
    typedef f32x16 T;
};

template <int S>
__device__ __forceinline__ typename MxAcc<S>::T mfma_bf16(bf16x8 r, bf16x8 c, typename MxAcc<S>::T acc)
{
    if constexpr (S == 16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(r, c, acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(r, c, acc, 0, 0, 0);
}

// Of an instruction's S x S sums a lane has S * S / 64: sum e is that of A's row `lane % S` and of B's row_of_sum<S>(e, lane / S).
template <int S>
__device__ __forceinline__ int row_of_sum(int e, int grp)
{
    return e / 4 * 8 + grp * 4 + e % 4;
}

// sum += the products of block b of S rows of A and of B: pa, sa, pb and sb are the codes and scales of this lane's row of each.
template <int FA, int FB, int S>
__device__ __forceinline__ void add_block(const uint8_t* pa, const uint8_t* sa, const uint8_t* pb, const uint8_t* sb, int64_t b,
                                          int grp, typename MxAcc<S>::T& sum)
{
    const int ea = sa[b], eb = sb[b];
    typename MxAcc<S>::T part{};
#pragma unroll
    for (int h = 0; h < S / 16; ++h) {
        const int p = h * (64 / S) + grp;
        part = mfma_bf16<S>(block8<FB>(pb, b, p), block8<FA>(pa, b, p), part);
    }
#pragma unroll
    for (int e = 0; e < S * S / 64; ++e) {
        const int ej = __shfl(eb, row_of_sum<S>(e, grp));
        sum[e] += ea == 255 || ej == 255 ? __builtin_nanf("") : ldexpf(part[e], ea + ej - 254);
    }
}

__device__ __forceinline__ bool no_number(float v) { return !(fabsf(v) < __builtin_inff()); }

}  // namespace fq
