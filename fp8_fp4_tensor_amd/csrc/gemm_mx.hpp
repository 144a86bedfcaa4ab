// gemm_mx.hpp -- the pieces of the product of MX planes: k_gemm_mx.hip chooses
// and launches; the tiles' kernels are compiled by A's format.
#pragma once

#include "launch.hpp"

namespace fq {

enum MxOut : int { kOutF32 = 0, kOutBf16, kOutPart };

struct MxTileArgs {
    GemmMxArgs g;
    // Scale words (those of 128 elements of a row), `words` of a row: as the
    // planes have them, or (arranged) row r's word i at word (r / 64 * words + i) * 64
    // + r % 64, as k_gemm_mx_scales lays them out.
    const uint32_t* sa = nullptr;
    const uint32_t* sb = nullptr;
    int words = 0;
    int arranged = 0;
    int tiles_m = 0, tiles_n = 0;
    int out = 0;             // MxOut
    float* part = nullptr;   // [gridDim.y, m, n] for kOutPart
};

// The tile kernels of plan.hpp's kind, over `splits` shares of k.
hipError_t launch_mx_tiles_e4m3(const MxTileArgs& x, int kind, int splits, hipStream_t stream);
hipError_t launch_mx_tiles_e5m2(const MxTileArgs& x, int kind, int splits, hipStream_t stream);
hipError_t launch_mx_tiles_e2m1(const MxTileArgs& x, int kind, int splits, hipStream_t stream);

}  // namespace fq
