// k_gemm_mx_e5m2.hip -- tiles of the product of MX planes whose A is E5M2.
#include "gemm_mx_tile.hpp"

namespace fq {

hipError_t launch_mx_tiles_e5m2(const MxTileArgs& x, int kind, int splits, hipStream_t st)
{
    return mx_launch<kE5M2>(x, kind, splits, st);
}

}  // namespace fq
