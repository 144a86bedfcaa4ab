// k_gemm_mx_e4m3.hip -- tiles of the product of MX planes whose A is E4M3.
#include "gemm_mx_tile.hpp"

namespace fq {

hipError_t launch_mx_tiles_e4m3(const MxTileArgs& x, int kind, int splits, hipStream_t st)
{
    return mx_launch<kE4M3>(x, kind, splits, st);
}

}  // namespace fq
