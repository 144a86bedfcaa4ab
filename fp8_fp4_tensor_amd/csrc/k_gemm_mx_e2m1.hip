// k_gemm_mx_e2m1.hip -- tiles of the product of MX planes whose A is E2M1.
#include "gemm_mx_tile.hpp"

namespace fq {

hipError_t launch_mx_tiles_e2m1(const MxTileArgs& x, int kind, int splits, hipStream_t st)
{
    return mx_launch<kE2M1>(x, kind, splits, st);
}

}  // namespace fq
