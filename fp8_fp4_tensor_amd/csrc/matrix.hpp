// matrix.hpp -- what the matrix products share on the device: operands as the
// 8- and 4-bit matrix instructions take them, transfers to LDS, the walk over
// tiles and the store of results.
#pragma once

#include "codec.hpp"

namespace fq {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

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
__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int64_t& tm, int64_t& tn)
{
    const uint32_t total = gridDim.x, per = total / 8, rest = total % 8;
    const uint32_t xcd = blockIdx.x % 8, nth = blockIdx.x / 8;
    const uint32_t t = xcd * per + min(xcd, rest) + nth;
    const uint32_t wide = 8 * (uint32_t)tiles_n;
    const uint32_t band = t / wide, in = t - band * wide;
    const uint32_t high = min(8u, (uint32_t)tiles_m - band * 8);
    tn = in / high;
    tm = band * 8 + (in - (uint32_t)tn * high);
}

}  // namespace fq
