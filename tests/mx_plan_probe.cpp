// The launch rule of products of microscaled operands, compiled without HIP, as
// functions a test can call.
#include "plan.hpp"

extern "C" void mx_plan(int64_t m, int64_t n, int64_t k, int64_t a4, int64_t b4, int64_t bf16, int64_t* out)
{
    const fq::MxPlan p = fq::plan_gemm_mx(m, n, k, a4 != 0, b4 != 0, bf16 != 0);
    out[0] = p.kind;
    out[1] = p.splits;
    out[2] = p.main;
    out[3] = p.arranged;
}

extern "C" void mx_tile_sizes(int64_t* out)
{
    for (int i = 0; i < fq::kMxTileKinds; ++i) {
        out[2 * i] = fq::kMxTiles[i].tm;
        out[2 * i + 1] = fq::kMxTiles[i].tn;
    }
}
