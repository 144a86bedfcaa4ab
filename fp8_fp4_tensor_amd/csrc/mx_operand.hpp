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

}  // namespace fq
