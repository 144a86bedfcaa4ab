// k_attn.hip -- attention over the paged 8-bit cache on gfx950.
//
//   s = scale * ks[block of t] * (q . K_t)      (then cap * tanh(s / cap))
//   o = sum_t p_t * vs[block of t] * V_t,  p = softmax of s over the visible t
//
// The codes become bf16 in registers (exact: both 8-bit formats are subsets
// of bf16) and meet bf16 queries in v_mfma_f32_16x16x32_bf16 (32x32x16 with
// many rows and at most 128 dims); the block scales multiply scores and probabilities in fp32. For the second product
// p * vs becomes bf16: with many rows one term, off by at most 2^-8 of each
// p, as the bf16 output's own rounding is of their sum; with few rows two
// terms, for there the matrix unit has time. The sum of the unrounded p, the
// maxima and the accumulators are fp32.
//
// Layout (32x32 tiles: see there): no operand crosses lanes. The first product computes S^T = K Q^T,
// K's tokens as the instruction's rows. A step takes 64 tokens as four row
// tiles; row r of tile n is token 16 (r / 4) + 4 n + r % 4, so that the four
// results a lane gets from each tile are, over the four tiles, 16
// consecutive tokens of one query row. Those are just what the second
// product O^T = V^T P^T wants from that lane as its column operand, and with
// V stored transposed (a head's page is [dim, page_tokens]) the same 16
// tokens of a value row are one 16-byte load. So a lane sees one block scale,
// one page and one query row a step; the row statistics are per-lane scalars,
// joined over the four lane groups by two exchanges.
#include "codec.hpp"
#include "launch.hpp"
#include "plan.hpp"

namespace fq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = kAttnStep;  // tokens a wave takes at once
constexpr int kRows = kAttnRows;  // query rows of a workgroup
constexpr int kMaxSplits = kAttnSplits;
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
// The least factor of a score: -inf times it is -inf, and the largest product
// times it 6e-5, a product of 1e33 2e-10. (2^-149 is an operand of four bytes
// less, and the code so placed 1.4% slower with 256 dims: 534 us for 527.)
constexpr float kLeast = 0x1p-142f;

// Eight codes -> eight bf16 (exact).
template <int FMT>
__device__ __forceinline__ bf16x8 widen8(uint32_t a, uint32_t b)
{
    bf16x2 r[4];
    if constexpr (FMT == kE4M3) {
        r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
        r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
        r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
        r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    } else {
        r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, 1.0f, false);
        r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, 1.0f, true);
        r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, 1.0f, false);
        r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, 1.0f, true);
    }
    return bf16x8{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

__device__ __forceinline__ f32x4 mfma(bf16x8 rows, bf16x8 cols, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(rows, cols, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mfma32(bf16x8 rows, bf16x8 cols, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(rows, cols, c, 0, 0, 0);
}

// The cap: a score s (base 2) becomes c2 tanh(y), y = s / c2, c2 = log2(e) cap.
// Near zero, for |y| <= 1/2, that is s times tanh(y) / y, a polynomial in y y
// (equal-ripple fit of four terms, off by 1.4e-8, in fp32 by less than a unit), so
// that the error is relative to the score however large the cap is. Further out
// it is c2 (1 - 2 / (e^2y + 1)), where a unit of c2 is at most 2.2 units of the
// result; the reciprocal is the instruction's, off by a unit. A wave whose scores
// are all near, as they are under the usual caps, skips the exponential and the
// reciprocal, 16 cycles each: 2 chunks of 2048 rows, 32 heads, up to 8192 keys take
// 441 us without a cap, 559 with all scores near and 610 where most are far.
constexpr float kCapNear = 0.5f;
__device__ __forceinline__ float cap_ratio(float yy)
{
    float p = 0.017256994f;
    p = __builtin_fmaf(yy, p, -0.053052951f);
    p = __builtin_fmaf(yy, p, 0.13325988f);
    p = __builtin_fmaf(yy, p, -0.33333150f);
    return __builtin_fmaf(yy, p, 1.0f);
}
__device__ __forceinline__ float soft_cap(float s, float c2, float inv)
{
    const float y = s * inv;
    const float far = __builtin_fmaf(-2.0f * c2, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(y * (2.0f * kLog2e)) + 1.0f), c2);
    return fabsf(y) <= kCapNear ? s * cap_ratio(y * y) : far;
}

// Max over the four lane groups (lanes l, l ^ 16, l ^ 32, l ^ 48), in every
// lane: the swaps exchange odd 16-lane rows with even ones, then the halves.
__device__ __forceinline__ float max_groups(float v)
{
    typedef uint32_t pair __attribute__((ext_vector_type(2)));
    const uint32_t b = __float_as_uint(v);
    const pair r = __builtin_bit_cast(pair, __builtin_amdgcn_permlane16_swap(b, b, false, false));
    const uint32_t c = __float_as_uint(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
    const pair h = __builtin_bit_cast(pair, __builtin_amdgcn_permlane32_swap(c, c, false, false));
    return fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
}

// Max over lanes l and l ^ 32, in both.
__device__ __forceinline__ float max_halves(float v)
{
    const uint32_t b = __float_as_uint(v);
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(b, b, false, false));
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The keys that the rows [r0, r1) of a sequence and head see: [lo, hi), empty
// if hi <= lo; from is lo rounded down to a step.
struct Span {
    int lo, hi, from;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const KvSeq& s, int r0, int r1, int group)
{
    Span p;
    const int first = s.len - s.nq;
    const int pos0 = first + r0 / group, pos1 = first + (r1 - 1) / group;  // r1 > r0
    p.hi = max(pos1 + 1, 0);
    p.lo = a.window > 0 ? max(pos0 - a.window + 1, 0) : 0;
    p.from = p.lo & ~(kStep - 1);
    return p;
}

// Four dims of an output row from its maximum (base 2), sum and accumulator. The
// sum is 0 for a row that sees nothing; a query that is no number gives a sum
// that is none.
__device__ __forceinline__ void finish(const AttnArgs& a, int64_t rid, int dim, int d, float top, float sum, f32x4 v)
{
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        b[e] = __builtin_bit_cast(uint16_t, (__bf16)(v[e] * inv));
    *(u32x2*)(a.out + rid * dim + d) = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
    if (a.lse && d == 0)
        a.lse[rid] = sum == 0.0f ? -kInf : (top + __log2f(sum)) * kLn2;
}

// Few query rows (one token of a grouped head, or short runs): the waves of a
// workgroup take the steps of a run of keys in turn and join their results in
// LDS. Bound by reading the cache once, that is by how much is under way: a
// wave fetches the next step's keys and values as soon as this step's scores
// are done (values have two sets of registers, keys one), and page indexes a
// step before that.
template <int D, int FMT, int kWaves, bool SPLIT>
__global__ __launch_bounds__(kWaves * 64, D <= 128 ? 2 : 1) void k_attn(AttnArgs a)
{
    constexpr int C = D / 64;  // 16-byte chunks of a key row a lane holds
    constexpr int T = D / 16;  // value row tiles
    __shared__ float lds_o[kWaves][kRows][D + 4];
    __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = lane & 15, grp = lane >> 4;
    const int group = a.q_heads / kv.heads;
    // heads run fastest: workgroups go round robin to the XCDs, so with eight
    // heads each XCD's L2 sees the keys and values of one of them
    const unsigned ht = blockIdx.x / (unsigned)kv.heads;
    const int h = (int)(blockIdx.x - ht * (unsigned)kv.heads);
    const int r0 = (int)(ht % (unsigned)a.tiles) * kRows;
    const int split = (int)(ht / (unsigned)a.tiles);
    const int seq = (int)blockIdx.y;
    const int32_t* table = kv.table + (int64_t)seq * kv.max_pages;
    const int ps = 31 - __clz(kv.page), bs = 31 - __clz(kv.block);
    int page_k = 0, page_v = 0;
    auto pages = [&](int t0) {  // held to the table's end
        page_k = table[min((t0 + (row >> 2) * 16) >> ps, kv.max_pages - 1)];
        page_v = table[min((t0 + grp * 16) >> ps, kv.max_pages - 1)];
    };
    // without a window the first step does not depend on the sequence's
    // length: its pages are looked up beside it, not after it
    if (a.window == 0 && kv.max_len > 0)
        pages(split * a.chunk + w * kStep);
    const KvSeq s = kv_seq(kv, seq);
    const int rows = s.nq * group;
    if (r0 >= rows)
        return;
    const Span sp = span_of(a, s, r0, min(r0 + kRows, rows), group);
    const int begin = sp.from + split * a.chunk;
    const int end = SPLIT ? min(sp.hi, begin + a.chunk) : sp.hi;
    if (SPLIT && begin >= end)
        return;

    const int r = min(r0 + row, rows - 1);  // rows past the last repeat it and are not stored
    const int tok = r / group, head = h * group + r % group;
    const int pos = s.len - s.nq + tok;
    const int oldest = a.window > 0 ? pos - a.window + 1 : -0x7fffffff;
    bf16x8 q[C][2];
    {
        const uint16_t* p = a.q + (s.q0 + tok) * a.q_stride + (int64_t)head * D + grp * 16;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            q[c][0] = __builtin_bit_cast(bf16x8, ld16(p + c * 64));
            q[c][1] = __builtin_bit_cast(bf16x8, ld16(p + c * 64 + 8));
        }
    }
    const float sc2 = a.scale * kLog2e;  // products to scores, base 2
    float m = -kInf, l = 0.0f;
    f32x4 o[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
        o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // A step's keys (row r: tokens 16 (r / 4) + 4 n + r % 4) and values (this
    // lane's 16 scored tokens), their scales and whether their page exists.
    struct Values {
        u32x4 c[T];
        float ks, vs;
        bool ok;
    };
    u32x4 kc[4][C];
    Values val[2];
    auto load = [&](int t0, Values& v) {
        const int tk = t0 + (row >> 2) * 16, tv = t0 + grp * 16;
        v.ok = page_v >= 0 && page_v < kv.num_pages;
        const int pk = page_k >= 0 && page_k < kv.num_pages ? page_k : 0, pv = v.ok ? page_v : 0;
        const uint8_t* kp =
            kv.k + (((int64_t)pk * kv.heads + h) * kv.page + (tk & (kv.page - 1)) + (row & 3)) * D + grp * 16;
        const int64_t vt = ((int64_t)pv * kv.heads + h) * kv.page;
        const uint8_t* vp = kv.v + vt * D + (int64_t)row * kv.page + (tv & (kv.page - 1));
        const int64_t blk = (vt >> bs) + ((tv & (kv.page - 1)) >> bs);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int c = 0; c < C; ++c)
                kc[n][c] = ld16(kp + n * 4 * D + c * 64);
        v.ks = kv.ks[blk];
        v.vs = kv.vs[blk];
        __builtin_amdgcn_sched_barrier(0);  // loads return in order: keys, which are used first, go first
#pragma unroll
        for (int t = 0; t < T; ++t)
            v.c[t] = ld16(vp + (int64_t)t * 16 * kv.page);
    };
    const int hop = kWaves * kStep;
    auto step = [&](int t0, Values& v, Values& next) {
        const int tv = t0 + grp * 16;
        float x[16];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                d = mfma(widen8<FMT>(kc[n][c][0], kc[n][c][1]), q[c][0], d);
                d = mfma(widen8<FMT>(kc[n][c][2], kc[n][c][3]), q[c][1], d);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[n * 4 + e] = d[e];
        }
        const float f = v.ks * sc2;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x[e] *= f;
        if (a.cap2 > 0.0f) {
            float most = fabsf(x[0]);
#pragma unroll
            for (int e = 1; e < 16; ++e)
                most = fmaxf(most, fabsf(x[e]));
            if (__all(most * a.cap_inv <= kCapNear)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float y = x[e] * a.cap_inv;
                    x[e] *= cap_ratio(y * y);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = soft_cap(x[e], a.cap2, a.cap_inv);
            }
        }
        const bool inside = t0 >= sp.lo && t0 + kStep <= end && v.ok && t0 + kStep - 1 <= pos && t0 >= oldest;
        if (!__all(inside)) {
            // scores of keys that a row does not see go to -inf; values of keys
            // that no row sees (a page's unused or outdated part) to zero, for
            // they may hold anything and 0 * NaN is not 0
            const int from = max(sp.lo - tv, 0), to = v.ok ? min(end - tv, 16) : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const bool see = e >= from && e < to && tv + e <= pos && tv + e >= oldest;
                x[e] = see ? x[e] : -kInf;
            }
            v.vs = from < to ? v.vs : 0.0f;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                uint32_t keep = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    keep |= (d * 4 + b >= from && d * 4 + b < to) ? 0xffu << (8 * b) : 0u;
#pragma unroll
                for (int t = 0; t < T; ++t)
                    v.c[t][d] &= keep;
            }
        }
        if (t0 + hop < end) {
            load(t0 + hop, next);
            pages(t0 + 2 * hop);
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 16; ++e)
            top = fmaxf(top, x[e]);
        top = max_groups(top);
        // m is a row's reference, not its exact maximum: it follows only where a
        // score passes it by more than 2^kSlack (and at a row's first score), so
        // that the accumulators are rarely touched between products. The
        // probabilities' sums stay below 2^kSlack per term, and rounding is
        // relative.
        if (__any(top > m + kSlack)) {
            const float mn = fmaxf(m, top);
            const float alpha = __builtin_amdgcn_exp2f(m - (mn == -kInf ? 0.0f : mn));
            m = mn;
            l *= alpha;
#pragma unroll
            for (int t = 0; t < T; ++t)
                o[t] *= alpha;
        }
        const float mu = m == -kInf ? 0.0f : m;  // a row that has seen nothing yet
        // p * vs in two bf16 terms: the second product costs twice its matrix
        // instructions, which reading the cache hides, and keeps 16 bits of p
        float sum = 0.0f;
        bf16x8 p[2], rest[2];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float f = __builtin_amdgcn_exp2f(x[e] - mu), y = f * v.vs;
            sum += f;
            p[e >> 3][e & 7] = (__bf16)y;
            rest[e >> 3][e & 7] = (__bf16)(y - (float)p[e >> 3][e & 7]);
        }
        l += sum;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const bf16x8 lo = widen8<FMT>(v.c[t][0], v.c[t][1]), hi = widen8<FMT>(v.c[t][2], v.c[t][3]);
            o[t] = mfma(lo, p[0], o[t]);
            o[t] = mfma(hi, p[1], o[t]);
            o[t] = mfma(lo, rest[0], o[t]);
            o[t] = mfma(hi, rest[1], o[t]);
        }
    };
    int t0 = begin + w * kStep;
    if (t0 < end) {
        if (a.window != 0)
            pages(t0);
        load(t0, val[0]);
        pages(t0 + hop);
    }
    while (t0 < end) {
        step(t0, val[0], val[1]);
        t0 += hop;
        if (t0 >= end)
            break;
        step(t0, val[1], val[0]);
        t0 += hop;
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (grp == 0) {
        lds_m[w][row] = m;
        lds_l[w][row] = l;
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
        *(f32x4*)&lds_o[w][row][t * 16 + grp * 4] = o[t];
    __syncthreads();
    // a thread takes four dims of a row at a time
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kWaves * 64) {
        const int orow = i / (D / 4), d = i % (D / 4) * 4;
        if (r0 + orow >= rows)
            break;
        float top = lds_m[0][orow];
#pragma unroll
        for (int k = 1; k < kWaves; ++k)
            top = fmaxf(top, lds_m[k][orow]);
        const float mu = top == -kInf ? 0.0f : top;
        float sum = 0.0f;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            const float f = __builtin_amdgcn_exp2f(lds_m[k][orow] - mu);
            sum += lds_l[k][orow] * f;
            v += *(const f32x4*)&lds_o[k][orow][d] * f;
        }
        const int ro = r0 + orow;
        const int64_t rid = (s.q0 + ro / group) * a.q_heads + h * group + ro % group;
        if constexpr (SPLIT) {
            // accumulators first, in whole 16 bytes, then the maxima and sums
            const int64_t at = rid * a.splits + split;
            if (d == 0)
                *(float2*)(a.ws + kv.total_q * a.q_heads * (int64_t)a.splits * D + at * 2) = make_float2(top, sum);
            *(f32x4*)(a.ws + at * D + d) = v;
        } else {
            finish(a, rid, D, d, top, sum, v);
        }
    }
}

// ---------------------------------------------------------------- many rows
// Prompts and chunks: a workgroup takes 8 waves of 32 query rows of one head
// group and walks over the keys in steps of 64. The step's codes are read once,
// widened to bf16 once, and shared in LDS, in two stages; the next step's are
// under way meanwhile and go to LDS between the second product's instructions.
// 32x32 tiles: the vector unit can issue beside a v_mfma_f32_32x32x16 for half
// of its cycles, beside a 16x16x32 not at all, and a lane has one query row to
// keep statistics of instead of two. A step of a wave is 32 matrix instructions
// (1024 cycles) and some 240 vector ones with 32 exponentials of 16 cycles
// (about 1400), of two waves a SIMD: bound by issuing both. 2 chunks of 2048
// rows, 32 heads over 8, up to 8192 keys: 435 to 448 us, about 985 TFLOP/s (474 with 16x16
// tiles; 393 without reading LDS, 400 without reading the cache, 375 without
// the softmax). Half a step's shift between the waves of a SIMD changed nothing.
//
// LDS rows: a token's dims (keys) or a dim's 64 tokens (values) in 16-byte
// chunks, turned so that reads of 16 bytes a lane meet no bank twice. The
// hardware serves 16 of 32 lanes at once, and the operand's rows that they read
// are all different modulo 16. `turn` is that number for LDS rows of 16 chunks
// (all banks), half of it for 8, where the row's parity picks the half of the
// banks itself.
template <int CHUNKS>
__device__ __forceinline__ int turn(int row)
{
    static_assert(CHUNKS == 8 || CHUNKS == 16, "64 or 128 dims, or 64 tokens");
    return CHUNKS == 8 ? row >> 1 & 7 : row & 15;
}
// The operand row (modulo 16) that token t is: see the step.
__device__ __forceinline__ int key_row(int t) { return (t & 3) | (t >> 2 & 4) | (t << 1 & 8); }

template <int D>
struct KvStage {
    uint16_t k[kStep * D], v[D * kStep];
};

template <int D, int FMT>
__global__ __launch_bounds__(512, 2) void k_attn_tile(AttnArgs a)
{
    static_assert(D <= 128, "256 dims: k_attn_tile256");
    constexpr int kTileRows = attn_tile_rows(D), kWaveRows = 32, kThreads = 512;
    constexpr int KK = D / 16, T = D / 32;
    constexpr int kLoads = 8 * D / kThreads;  // 16-byte chunks of codes a thread brings for a step
    __shared__ KvStage<D> stage[2];
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 31, half = lane >> 5;
    const int group = a.q_heads / kv.heads;
    const unsigned ht = blockIdx.x / (unsigned)kv.heads;
    const int h = (int)(blockIdx.x - ht * (unsigned)kv.heads);
    const int r0 = (a.tiles - 1 - (int)ht) * kTileRows;  // the last rows see the most keys: they start first
    const int seq = (int)blockIdx.y;
    const KvSeq s = kv_seq(kv, seq);
    const int rows = s.nq * group;
    if (r0 >= rows)
        return;
    const Span sp = span_of(a, s, r0, min(r0 + kTileRows, rows), group);
    // this wave's rows; a wave past the last row does the last row's work and stores nothing
    const int w0 = min(r0 + w * kWaveRows, rows - 1);
    const Span ws = span_of(a, s, w0, min(w0 + kWaveRows, rows), group);
    const int32_t* table = kv.table + (int64_t)seq * kv.max_pages;
    const int ps = 31 - __clz(kv.page), bs = 31 - __clz(kv.block), pm = kv.page - 1;

    bf16x8 q[KK];
    const int r = min(w0 + row, rows - 1);
    const int pos = s.len - s.nq + r / group;
    const int oldest = a.window > 0 ? pos - a.window + 1 : -0x7fffffff;
    {
        const uint16_t* p = a.q + (s.q0 + r / group) * a.q_stride + (int64_t)(h * group + r % group) * D + half * 8;
        // a negative scale turns the queries' signs, so that scores rise with their products
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int k = 0; k < KK; ++k)
            q[k] = __builtin_bit_cast(bf16x8, ld16(p + k * 16) ^ u32x4{flip, flip, flip, flip});
    }
    const float sc2 = fabsf(a.scale) * kLog2e;  // products to scores, base 2

    float m = -kInf, l = 0.0f;
    f32x16 o[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[t][e] = 0.0f;

    // A step's codes on their way: chunk i of this thread is of the keys
    // (token, 16 dims) below 4 D, of the values (dim, 16 tokens) above. A lane
    // looks up the page of tokens 16 (lane % 4) .. + 15, a step before: those of
    // its values and of a scale that it brings, the keys' for lane / 4 even, else
    // the values'. Its chunks of keys are of one page in the whole wave.
    u32x4 code[kLoads];
    float scale_next = 0.0f;
    bool ok_next = false;
    int page;
    const int mine = (lane & 3) * 16;
    const float* const scales = lane & 4 ? kv.vs : kv.ks;
    auto of_keys = [&](int i) { return kLoads > 1 ? i < kLoads / 2 : w < 4; };
    auto look_up = [&](int t0) { page = table[min((t0 + mine) >> ps, kv.max_pages - 1)]; };  // held to the table's end
    // a page's bytes (at most 2^28) and scales
    const uint32_t page_bytes = (uint32_t)kv.heads * kv.page * D, page_blocks = (uint32_t)kv.heads * kv.page >> bs;
    auto fetch = [&](int t0) {
        ok_next = (uint32_t)page < (uint32_t)kv.num_pages;
        const uint32_t held = ok_next ? (uint32_t)page : 0u;
        const int tv = (t0 + mine) & pm;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = threadIdx.x + i * kThreads;
            if (of_keys(i)) {
                const int t = c / (D / 16);
                const uint32_t p = __builtin_amdgcn_readlane(held, __builtin_amdgcn_readfirstlane(t >> 4));
                code[i] = ld16(kv.k + (uint64_t)p * page_bytes +
                               (uint32_t)((h * kv.page + ((t0 + t) & pm)) * D + c % (D / 16) * 16));
            } else {
                const uint8_t* from = kv.v + (uint32_t)((h * D + ((c - 4 * D) >> 2)) * kv.page);
                code[i] = ld16(from + (uint64_t)held * page_bytes + (uint32_t)tv);
            }
        }
        scale_next = scales[held * page_blocks + ((uint32_t)(h * kv.page + tv) >> bs)];  // one of at most 2^26
    };
    // The codes on their way -> a stage: first values that no row sees go to
    // zero, for they may hold anything, and 0 * NaN is not 0; then chunk by chunk.
    auto clear = [&](int t0) {
        const int t = t0 + mine;
        const int from = max(sp.lo - t, 0), end = ok_next ? min(sp.hi - t, 16) : 0;
        if (__all(from == 0 && end == 16))
            return;
        uint32_t keep[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            keep[e] = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                keep[e] |= (e * 4 + b >= from && e * 4 + b < end) ? 0xffu << (8 * b) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                code[i][e] &= of_keys(i) ? ~0u : keep[e];
    };
    int to[kLoads][2];  // where this thread's chunks go in a stage
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int c = threadIdx.x + i * kThreads, t = c / (D / 16), d = (c - 4 * D) >> 2;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            to[i][k] = of_keys(i) ? t * D + ((c % (D / 16) * 2 + k) ^ turn<D / 8>(key_row(t))) * 8
                                 : kStep * D + d * kStep + (((c & 3) * 2 + k) ^ turn<8>(d)) * 8;
    }
    auto put = [&](KvStage<D>& st, int i, int k) {
        *(bf16x8*)(st.k + to[i][k]) = widen8<FMT>(code[i][2 * k], code[i][2 * k + 1]);
    };

    // The first product's row r of tile n is token 32 n + 16 (r / 4 % 2) +
    // 4 (r / 8) + r % 4, so that a lane's 16 results are consecutive tokens of
    // one query row, and the first and last eight of them are just the column
    // operand of two of the second product's instructions.
    const int krow = (row >> 2 & 1) * 16 + (row >> 3) * 4 + (row & 3);
    auto step = [&](const KvStage<D>& st, KvStage<D>& next, int t0, float sc, uint64_t oks) {
        const float kf[2] = {__shfl(sc, half), __shfl(sc, half + 2)};
        const float vf[2] = {__shfl(sc, half + 4), __shfl(sc, half + 6)};
        // The operands of the next four instructions are read during these
        // four; fences keep the compiler from moving the reads to their use.
        bf16x8 fa[4], fb[4];
        auto keys = [&](bf16x8* to, int at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = (at + i) >> 1, n = i & 1;
                to[i] = *(const bf16x8*)(st.k + (n * 32 + krow) * D + ((k * 2 + half) ^ turn<D / 8>(row)) * 8);
            }
        };
        auto values = [&](bf16x8* to, int at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = (at + i) % T * 32 + row, k = (at + i) / T;
                to[i] = *(const bf16x8*)(st.v + d * kStep + (((k >> 1) * 4 + half * 2 + (k & 1)) ^ turn<8>(d)) * 8);
            }
        };
        f32x16 x[2];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[n][e] = 0.0f;
        keys(fa, 0);
#pragma unroll
        for (int g = 0; g < KK / 2; ++g) {
            if (g + 1 < KK / 2)
                keys(fb, (g + 1) * 4);
            else
                values(fb, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i & 1] = mfma32(fa[i], q[g * 2 + (i >> 1)], x[i & 1]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                fa[i] = fb[i];
        }
        // scores stay products until the exponential: x f - m is one fused
        // operation, and with f >= 0 the largest x has the largest score
        // (f > 0 also where no token of the group is seen and its scale may be
        // anything: a hidden score is -inf times f)
        const bool inside = t0 >= sp.lo && t0 + kStep <= sp.hi && (oks & 15) == 15 && t0 + kStep - 1 <= pos && t0 >= oldest;
        float f[2] = {kf[0], kf[1]};
        if (a.cap2 > 0.0f) {
            float most = 0.0f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float v = fabsf(x[n][0]);
#pragma unroll
                for (int e = 1; e < 16; ++e)
                    v = fmaxf(v, fabsf(x[n][e]));
                most = fmaxf(most, v * f[n]);
            }
            if (__all(most * a.cap_inv <= kCapNear)) {  // still products, and f their factor
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float g = fminf(f[n] * a.cap_inv, kFLT_MAX);  // finite, so that 0 stays 0
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float y = x[n][e] * g;
                        x[n][e] *= cap_ratio(y * y);
                    }
                }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[n][e] = soft_cap(x[n][e] * f[n], a.cap2, a.cap_inv);
                    f[n] = 1.0f;
                }
            }
        }
        if (!__all(inside)) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const bool ok = oks >> (half + 2 * n) & 1;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int t = t0 + n * 32 + half * 16 + e;
                    x[n][e] = ok && t >= sp.lo && t < sp.hi && t <= pos && t >= oldest ? x[n][e] : -kInf;
                }
            }
        }
        float top = -kInf;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float v = x[n][0];
#pragma unroll
            for (int e = 1; e < 16; ++e)
                v = fmaxf(v, x[n][e]);
            top = fmaxf(top, v == -kInf ? -kInf : v * f[n]);
        }
        top = max_halves(top);
        if (__any(top > m + kSlack)) {  // as in k_attn
            const float mn = fmaxf(m, top);
            const float alpha = __builtin_amdgcn_exp2f(m - (mn == -kInf ? 0.0f : mn));
            m = mn;
            l *= alpha;
#pragma unroll
            for (int t = 0; t < T; ++t)
                o[t] *= alpha;
        }
        bf16x8 p[4];
        const float mu = m == -kInf ? 0.0f : m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][e], f[n], -mu));
                sum[e & 3] += y;
                p[n * 2 + (e >> 3)][e & 7] = (__bf16)(y * vf[n]);
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        clear(t0 + kStep);
#pragma unroll
        for (int g = 0; g < T; ++g) {
            if (g + 1 < T)
                values(fb, (g + 1) * 4);
            constexpr int kPer = kLoads * 2 / T < 1 ? 1 : kLoads * 2 / T;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[(g * 4 + i) % T] = mfma32(fa[i], p[(g * 4 + i) / T], o[(g * 4 + i) % T]);
#pragma unroll
            for (int i = g * kPer; i < (g + 1) * kPer; ++i)
                put(next, i >> 1, i & 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                fa[i] = fb[i];
        }
    };
    // What a step needs of this lane's scale: of a key block, times the scores'
    // scale; of a value block, zero where no row sees its tokens, for it may be anything.
    auto factor = [&](int t0) {
        const int tv = t0 + mine;
        const float v = ok_next && tv < sp.hi && tv + 16 > sp.lo ? scale_next : 0.0f;
        const float k = scale_next * sc2;
        return lane & 4 ? v : fmaxf(k, kLeast);
    };

    if (sp.from < sp.hi) {
        look_up(sp.from);
        fetch(sp.from);
        look_up(sp.from + kStep);
        clear(sp.from);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                put(stage[0], i, k);
        float sc = factor(sp.from);
        uint64_t oks = __ballot(ok_next);
        int cur = 0;
        for (int t0 = sp.from; t0 < sp.hi; t0 += kStep) {
            __syncthreads();  // the step's stage is written, the other one read
            // (past the last step these fetch once more, unused: a branch
            // around them makes the compiler wait for them before the step)
            fetch(t0 + kStep);
            look_up(t0 + 2 * kStep);
            if (t0 < ws.hi && t0 + kStep > ws.lo) {
                step(stage[cur], stage[cur ^ 1], t0, sc, oks);
            } else {  // none of this wave's rows sees these keys
                clear(t0 + kStep);
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        put(stage[cur ^ 1], i, k);
            }
            sc = factor(t0 + kStep);
            oks = __ballot(ok_next);
            cur ^= 1;
        }
    }
    l += __shfl_xor(l, 32);
    if (r0 + w * kWaveRows + row < rows) {
        const int64_t rid = (s.q0 + r / group) * a.q_heads + h * group + r % group;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                finish(a, rid, D, t * 32 + i * 8 + half * 4, m, l,
                       f32x4{o[t][i * 4], o[t][i * 4 + 1], o[t][i * 4 + 2], o[t][i * 4 + 3]});
    }
}

// The same for 256 dims, whose accumulators leave no room for 32 rows a wave
// at two waves a SIMD: 16 rows a wave and 16x16 tiles (2 chunks of 2048 rows, 16
// heads over 4, up to 8192 keys: 527 us; 32x32 tiles with one wave a SIMD 627).
// Score tiles as in k_attn, one block of 16 tokens a lane; tokens 16 g + 8 k
// .. + 7 of a dim are chunk g + 4 k, so that a read meets no bank twice.
__device__ __forceinline__ int key_turn256(int t) { return (t & 3) | (t >> 2 & 12); }

template <int FMT>
__global__ __launch_bounds__(512, 2) void k_attn_tile256(AttnArgs a)
{
    constexpr int D = 256, kTileRows = attn_tile_rows(D), kWaveRows = 16;
    constexpr int KK = D / 32, T = D / 16;
    constexpr int kLoads = D / 64;  // 16-byte chunks of codes a thread brings for a step
    __shared__ KvStage<D> stage[2];
    const KvArgs& kv = a.kv;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = lane & 15, grp = lane >> 4;
    const int group = a.q_heads / kv.heads;
    const unsigned ht = blockIdx.x / (unsigned)kv.heads;
    const int h = (int)(blockIdx.x - ht * (unsigned)kv.heads);
    const int r0 = (a.tiles - 1 - (int)ht) * kTileRows;  // the last rows see the most keys: they start first
    const int seq = (int)blockIdx.y;
    const KvSeq s = kv_seq(kv, seq);
    const int rows = s.nq * group;
    if (r0 >= rows)
        return;
    const Span sp = span_of(a, s, r0, min(r0 + kTileRows, rows), group);
    // this wave's rows; a wave past the last row does the last row's work and stores nothing
    const int w0 = min(r0 + w * kWaveRows, rows - 1);
    const Span ws = span_of(a, s, w0, min(w0 + kWaveRows, rows), group);
    const int32_t* table = kv.table + (int64_t)seq * kv.max_pages;
    const int ps = 31 - __clz(kv.page), bs = 31 - __clz(kv.block), pm = kv.page - 1;

    bf16x8 q[KK];
    const int r = min(w0 + row, rows - 1);
    const int pos = s.len - s.nq + r / group;
    const int oldest = a.window > 0 ? pos - a.window + 1 : -0x7fffffff;
    {
        const uint16_t* p = a.q + (s.q0 + r / group) * a.q_stride + (int64_t)(h * group + r % group) * D + grp * 8;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int k = 0; k < KK; ++k)
            q[k] = __builtin_bit_cast(bf16x8, ld16(p + k * 32) ^ u32x4{flip, flip, flip, flip});
    }
    const float sc2 = fabsf(a.scale) * kLog2e;  // products to scores, base 2

    float m = -kInf, l = 0.0f;
    f32x4 o[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
        o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // A step's codes on their way: chunk i of this thread is of the keys
    // (token, 16 dims) below 4 D, of the values (dim, 16 tokens) above.
    // Page indexes are looked up a step before that.
    u32x4 code[kLoads];
    float ks_next = 0.0f, vs_next = 0.0f;
    bool ok_next = false, there[kLoads];
    int page[kLoads], page_s;
    auto token_of = [&](int i) {
        const int c = threadIdx.x + i * 512;
        return c < 4 * D ? c / (D / 16) : (c & 3) * 16;
    };
    auto pages = [&](int t0) {  // held to the table's end
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            page[i] = table[min((t0 + token_of(i)) >> ps, kv.max_pages - 1)];
        page_s = table[min((t0 + grp * 16) >> ps, kv.max_pages - 1)];
    };
    // What an address takes beyond the page: a page's bytes, and this thread's
    // place in it but for the token (a page holds at most 2^28 bytes of codes).
    const uint32_t page_bytes = (uint32_t)kv.heads * kv.page * D, page_blocks = (uint32_t)kv.heads * kv.page >> bs;
    const uint8_t* home[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int c = threadIdx.x + i * 512;
        home[i] = c < 4 * D ? kv.k + (uint32_t)(h * kv.page * D + c % (D / 16) * 16)
                            : kv.v + (uint32_t)(h * kv.page * D + ((c - 4 * D) >> 2) * kv.page);
    }
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = threadIdx.x + i * 512, t = (t0 + token_of(i)) & pm;
            there[i] = (uint32_t)page[i] < (uint32_t)kv.num_pages;
            code[i] = ld16(home[i] + (uint64_t)(there[i] ? (uint32_t)page[i] : 0u) * page_bytes +
                           (uint32_t)(c < 4 * D ? t * D : t));
        }
        ok_next = (uint32_t)page_s < (uint32_t)kv.num_pages;
        // at most 2^26 scales
        const uint32_t blk = (ok_next ? (uint32_t)page_s : 0u) * page_blocks +
                             ((uint32_t)(h * kv.page + ((t0 + grp * 16) & pm)) >> bs);
        ks_next = kv.ks[blk];
        vs_next = kv.vs[blk];
    };
    auto put = [&](KvStage<D>& st, int t0) {
        const bool whole = t0 >= sp.lo && t0 + kStep <= sp.hi;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = threadIdx.x + i * 512;
            u32x4 x = code[i];
            uint16_t* to;
            int at, hop, sw;  // its two chunks and their turn
            if (c < 4 * D) {
                const int t = c / (D / 16);
                to = st.k + t * D;
                at = c % (D / 16) * 2;
                hop = 1;
                sw = key_turn256(t);
            } else {
                const int d = (c - 4 * D) >> 2, t = t0 + (c & 3) * 16;
                to = st.v + d * kStep;
                at = c & 3;
                hop = 4;
                sw = d & 7;
                // values that no row sees go to zero: they may hold anything, and 0 * NaN is not 0
                if (!whole || !there[i]) {
                    const int from = max(sp.lo - t, 0), end = there[i] ? min(sp.hi - t, 16) : 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t keep = 0;
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            keep |= (e * 4 + b >= from && e * 4 + b < end) ? 0xffu << (8 * b) : 0u;
                        x[e] &= keep;
                    }
                }
            }
            *(bf16x8*)(to + (at ^ sw) * 8) = widen8<FMT>(x[0], x[1]);
            *(bf16x8*)(to + ((at + hop) ^ sw) * 8) = widen8<FMT>(x[2], x[3]);
        }
    };

    auto step = [&](const KvStage<D>& st, int t0, float ks, float vs, bool ok) {
        if (t0 >= ws.hi || t0 + kStep <= ws.lo)
            return;  // none of this wave's rows sees these keys
        const int tv = t0 + grp * 16;
        f32x4 x[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int t = (row >> 2) * 16 + n * 4 + (row & 3);
            x[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KK; ++k)
                x[n] = mfma(*(const bf16x8*)(st.k + t * D + ((k * 4 + grp) ^ key_turn256(t)) * 8), q[k], x[n]);
        }
        float f = fmaxf(ks * sc2, kLeast);
        const bool inside = t0 >= sp.lo && t0 + kStep <= sp.hi && ok && t0 + kStep - 1 <= pos && t0 >= oldest;
        if (a.cap2 > 0.0f) {  // as in k_attn_tile
            float most = fabsf(x[0][0]);
#pragma unroll
            for (int e = 1; e < 16; ++e)
                most = fmaxf(most, fabsf(x[e >> 2][e & 3]));
            if (__all(most * f * a.cap_inv <= kCapNear)) {
                const float g = fminf(f * a.cap_inv, kFLT_MAX);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float y = x[e >> 2][e & 3] * g;
                    x[e >> 2][e & 3] *= cap_ratio(y * y);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e >> 2][e & 3] = soft_cap(x[e >> 2][e & 3] * f, a.cap2, a.cap_inv);
                f = 1.0f;
            }
        }
        if (!__all(inside)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = tv + e;
                const bool see = ok && t >= sp.lo && t < sp.hi && t <= pos && t >= oldest;
                x[e >> 2][e & 3] = see ? x[e >> 2][e & 3] : -kInf;
            }
        }
        float top = x[0][0];
#pragma unroll
        for (int e = 1; e < 16; ++e)
            top = fmaxf(top, x[e >> 2][e & 3]);
        top = max_groups(top == -kInf ? -kInf : top * f);
        if (__any(top > m + kSlack)) {
            const float mn = fmaxf(m, top);
            const float alpha = __builtin_amdgcn_exp2f(m - (mn == -kInf ? 0.0f : mn));
            m = mn;
            l *= alpha;
#pragma unroll
            for (int t = 0; t < T; ++t)
                o[t] *= alpha;
        }
        bf16x8 p[2];
        const float mu = m == -kInf ? 0.0f : m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e >> 2][e & 3], f, -mu));
            sum[e & 3] += y;
            p[e >> 3][e & 7] = (__bf16)(y * vs);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int d = t * 16 + row;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                o[t] = mfma(*(const bf16x8*)(st.v + d * kStep + ((grp + 4 * k) ^ (d & 7)) * 8), p[k], o[t]);
        }
    };

    if (sp.from < sp.hi) {
        pages(sp.from);
        fetch(sp.from);
        pages(sp.from + kStep);
        put(stage[0], sp.from);
        float ks = ks_next, vs = vs_next;
        bool ok = ok_next;
        int cur = 0;
        for (int t0 = sp.from; t0 < sp.hi; t0 += kStep) {
            __syncthreads();  // the step's stage is written, the other one read
            // (past the last step these fetch once more, unused: a branch
            // around them makes the compiler wait for them before the step)
            fetch(t0 + kStep);
            pages(t0 + 2 * kStep);
            // a group of tokens that no row sees has a scale that may be anything
            const int tv = t0 + grp * 16;
            step(stage[cur], t0, ks, ok && tv < sp.hi && tv + 16 > sp.lo ? vs : 0.0f, ok);
            put(stage[cur ^ 1], t0 + kStep);
            ks = ks_next;
            vs = vs_next;
            ok = ok_next;
            cur ^= 1;
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (r0 + w * kWaveRows + row < rows) {
        const int64_t rid = (s.q0 + r / group) * a.q_heads + h * group + r % group;
#pragma unroll
        for (int t = 0; t < T; ++t)
            finish(a, rid, D, t * 16 + grp * 4, m, l, o[t]);
    }
}

// Joins the partial results of a row's splits: a workgroup a row. The splits'
// maxima and sums are read side by side; then kParts groups of D / 4 threads
// add up every kParts-th split's four dims and meet in LDS, in order.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a)
{
    constexpr int kCols = D / 4, kParts = 256 / kCols;
    __shared__ float factor[kMaxSplits];
    __shared__ f32x4 part[kParts][kCols];
    __shared__ float red[8];
    const KvArgs& kv = a.kv;
    const int group = a.q_heads / kv.heads;
    const KvSeq s = kv_seq(kv, (int)blockIdx.y);
    const unsigned at = blockIdx.x / (unsigned)kv.heads;
    const int ro = (int)at, h = (int)(blockIdx.x - at * (unsigned)kv.heads), rows = s.nq * group;
    if (ro >= rows)
        return;
    const int r0 = ro / kRows * kRows;
    const Span sp = span_of(a, s, r0, min(r0 + kRows, rows), group);
    const int n = sp.hi > sp.from ? (int)cdiv(sp.hi - sp.from, a.chunk) : 0;
    const int64_t rid = (s.q0 + ro / group) * a.q_heads + h * group + ro % group;
    const float* from = a.ws + rid * a.splits * D;
    const float2* ml = (const float2*)(a.ws + kv.total_q * a.q_heads * (int64_t)a.splits * D) + rid * a.splits;
    const int w = threadIdx.x >> 6;
    float2 v[kMaxSplits / 256];
    float top = -kInf;
#pragma unroll
    for (int k = 0; k < kMaxSplits / 256; ++k) {
        const int i = threadIdx.x + k * 256;
        v[k] = i < n ? ml[i] : make_float2(-kInf, 0.0f);
        top = fmaxf(top, v[k].x);
    }
    top = max_workgroup(top, red);
    const float mu = top == -kInf ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxSplits / 256; ++k) {
        const int i = threadIdx.x + k * 256;
        const float f = __builtin_amdgcn_exp2f(v[k].x - mu);
        sum += v[k].y * f;
        if (i < n)
            factor[i] = f;
    }
#pragma unroll
    for (int x = 1; x < 64; x *= 2)
        sum += __shfl_xor(sum, x);
    if ((threadIdx.x & 63) == 0)
        red[4 + w] = sum;
    __syncthreads();
    sum = (red[4] + red[5]) + (red[6] + red[7]);
    const int col = threadIdx.x % kCols, p = threadIdx.x / kCols;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = p; i < n; i += kParts)
        o += *(const f32x4*)(from + (int64_t)i * D + col * 4) * factor[i];
    part[p][col] = o;
    __syncthreads();
    if (p > 0)
        return;
#pragma unroll
    for (int x = 1; x < kParts; ++x)
        o += part[x][col];
    finish(a, rid, D, col * 4, top, sum, o);
}

template <int D, int FMT>
hipError_t run(const AttnArgs& a, hipStream_t st)
{
    if (a.rows > kRows) {
        const dim3 tiles((unsigned)(a.tiles * a.kv.heads), (unsigned)a.kv.batch);
        if constexpr (D == 256)
            k_attn_tile256<FMT><<<tiles, 512, 0, st>>>(a);
        else
            k_attn_tile<D, FMT><<<tiles, 512, 0, st>>>(a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((int64_t)a.splits * a.tiles * a.kv.heads), (unsigned)a.kv.batch);
    if (a.splits == 1) {
        if (D <= 128 && a.waves == 8)
            k_attn<D, FMT, D <= 128 ? 8 : 4, false><<<grid, 512, 0, st>>>(a);
        else
            k_attn<D, FMT, 4, false><<<grid, 256, 0, st>>>(a);
        return hipGetLastError();
    }
    k_attn<D, FMT, 4, true><<<grid, 256, 0, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const dim3 jgrid((unsigned)((int64_t)a.kv.max_q * a.q_heads), (unsigned)a.kv.batch);
    k_attn_join<D><<<jgrid, 256, 0, st>>>(a);
    return hipGetLastError();
}

template <int D>
hipError_t by_format(const AttnArgs& a, hipStream_t st)
{
    return a.kv.fmt == kE4M3 ? run<D, kE4M3>(a, st) : run<D, kE5M2>(a, st);
}

}  // namespace

size_t plan_attention(AttnArgs& a)
{
    const KvArgs& kv = a.kv;
    const AttnPlan p = plan_attention(kv.batch, kv.heads, a.q_heads, kv.dim, kv.max_q, kv.max_len, a.window);
    a.rows = p.rows;
    a.tiles = p.tiles;
    a.waves = p.waves;
    a.chunk = p.chunk;
    a.splits = p.splits;
    return p.splits > 1 ? (size_t)(kv.total_q * a.q_heads) * p.splits * (kv.dim + 2) * sizeof(float) : 0;
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t st)
{
    switch (a.kv.dim) {
    case 64: return by_format<64>(a, st);
    case 128: return by_format<128>(a, st);
    default: return by_format<256>(a, st);
    }
}

}  // namespace fq
