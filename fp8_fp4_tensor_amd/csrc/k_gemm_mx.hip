// k_gemm_mx.hip -- the matrix product of MX planes on gfx950.
//
//   C[i, j] = sum_b 2^(ea[i, b] - 127) 2^(eb[j, b] - 127) sum_{t < 32} A[i, 32 b + t] B[j, 32 b + t]
//
// A: [m, k] and B: [n, k] codes, E4M3, E5M2 or E2M1 on either side, with one
// E8M0 code for 32 elements of a row. Both run along k, and the matrix
// instruction applies the scales, so a product is nothing but operands in and
// sums out.
//
// Operand order: B's rows are the instruction's rows and A's rows its columns,
// so a lane holds one row i of C and four consecutive columns j.
#include "launch.hpp"
#include "mx_operand.hpp"

namespace fq {
namespace {

// One workgroup computes 16x16 outputs; its waves take pairs of 128 elements
// of k in turn and their sums meet in LDS, in wave order.
constexpr int kFewWaves = 8;

// The operand of a lane: 128 elements from element k0 of the row at p, zeros past k.
template <int F, bool WIDE>
__device__ __forceinline__ i32x8 load128(const uint8_t* p, int64_t k0, int64_t k, int g, bool stream)
{
    const u32x4 zero = {0u, 0u, 0u, 0u};
    auto ld = [&](int64_t at) { return stream ? ld16_stream(p + at) : ld16(p + at); };
    if constexpr (F == kE2M1) {
        const int64_t at = k0 + 32 * g;
        return join(at < k ? ld(at >> 1) : zero, zero);
    } else {
        // widened: whole blocks, as a 4-bit side has them
        const int64_t lo = k0 + (WIDE ? 32 * g : 16 * g), hi = WIDE ? lo + 16 : lo + 64;
        return join(lo < k ? ld(lo) : zero, hi < k ? ld(hi) : zero);
    }
}

template <int FA, int FB, bool F32>
__global__ __launch_bounds__(kFewWaves * 64) void k_gemm_mx_few(GemmMxArgs a)
{
    constexpr bool WIDE = kWidened<FA, FB, F32>;
    __shared__ f32x4 part[kFewWaves][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16;
    const int64_t nb = a.k >> 5;
    // rows and columns past the last repeat it and are not stored
    const int64_t i = min(m0 + row, a.m - 1), j = min(n0 + row, a.n - 1);
    const uint8_t* pa = a.a + mx_bytes<FA>(i * a.k);
    const uint8_t* pb = a.b + mx_bytes<FB>(j * a.k);
    const uint8_t* psa = a.sa + i * nb;
    const uint8_t* psb = a.sb + j * nb;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t k0 = 256 * w; k0 < a.k; k0 += 256 * kFewWaves) {
        i32x8 fa[2], fb[2];
        uint32_t sa[2], sb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t b = min((k0 + 128 * h) / 32 + g, nb - 1);
            fb[h] = load128<FB, WIDE>(pb, k0 + 128 * h, a.k, g, true);
            fa[h] = load128<FA, WIDE>(pa, k0 + 128 * h, a.k, g, false);
            sb[h] = psb[b];
            sa[h] = psa[b];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (WIDE) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<FB>(fb[h], e, e8m0_value(sb[h])),
                                                                  widen8<FA>(fa[h], e, e8m0_value(sa[h])), acc, 0, 0, 0);
            } else {
                acc = mfma_mx<FB, FA>(fb[h], sb[h], fa[h], sa[h], acc);
            }
        }
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w > 0 || m0 + row >= a.m)
        return;
#pragma unroll
    for (int x = 1; x < kFewWaves; ++x)
        acc += part[x][lane];
    store4<!F32>(a.c, m0 + row, n0 + g * 4, a.n, acc, a.acc);
}

template <int FA, int FB>
hipError_t few(const GemmMxArgs& a, hipStream_t st)
{
    const dim3 grid((unsigned)cdiv(a.n, 16), (unsigned)cdiv(a.m, 16));
    constexpr int th = kFewWaves * 64;
    a.bf ? k_gemm_mx_few<FA, FB, false><<<grid, th, 0, st>>>(a) : k_gemm_mx_few<FA, FB, true><<<grid, th, 0, st>>>(a);
    return hipGetLastError();
}

template <int FA>
hipError_t with_b(const GemmMxArgs& a, hipStream_t st)
{
    return a.fb == kE4M3 ? few<FA, kE4M3>(a, st) : a.fb == kE5M2 ? few<FA, kE5M2>(a, st) : few<FA, kE2M1>(a, st);
}

}  // namespace

size_t gemm_mx_workspace(const GemmMxArgs&) { return 0; }

hipError_t launch_gemm_mx(const GemmMxArgs& a, hipStream_t st)
{
    if (a.k == 0) {
        GemmArgs g;
        g.m = a.m;
        g.n = a.n;
        g.c = a.c;
        g.bf = a.bf;
        g.acc = a.acc;
        return launch_gemm_join(g, 0, st);
    }
    return a.fa == kE4M3 ? with_b<kE4M3>(a, st) : a.fa == kE5M2 ? with_b<kE5M2>(a, st) : with_b<kE2M1>(a, st);
}

}  // namespace fq
