// The launch rules of the operators on 8-bit data, compiled without HIP, as
// functions a test can call.
#include "plan.hpp"

extern "C" void gemm_plan(int64_t m, int64_t n, int64_t k, int bf16, int64_t* out)
{
    const fq::GemmPlan p = fq::plan_gemm(m, n, k, bf16 != 0);
    out[0] = p.kind;
    out[1] = p.splits;
    out[2] = p.main;
}

extern "C" void attention_plan(int64_t batch, int64_t heads, int64_t q_heads, int dim, int64_t max_q, int64_t max_len,
                               int64_t window, int64_t* out)
{
    const fq::AttnPlan p = fq::plan_attention(batch, heads, q_heads, dim, max_q, max_len, window);
    out[0] = p.rows;
    out[1] = p.waves;
    out[2] = p.splits;
    out[3] = p.chunk;
    out[4] = p.tiles;
}

extern "C" void tile_sizes(int64_t* out)
{
    for (int i = 0; i < fq::kTileKinds; ++i) {
        out[2 * i] = fq::kTileCosts[i].tm;
        out[2 * i + 1] = fq::kTileCosts[i].tn;
    }
}
