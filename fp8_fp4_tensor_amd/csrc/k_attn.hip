// k_attn.hip -- attention over the paged 8-bit cache on gfx950.
//
//   s = scale * ks[block of t] * (q . K_t)      (then cap * tanh(s / cap))
//   o = sum_t p_t * vs[block of t] * V_t,  p = softmax of s over the visible t
//
// The codes become bf16 in registers (exact: both 8-bit formats are subsets
// of bf16) and meet bf16 queries in v_mfma_f32_16x16x32_bf16; the block
// scales multiply scores and probabilities in fp32. For the second product
// p * vs becomes bf16: with many rows one term, off by at most 2^-8 of each
// p, as the bf16 output's own rounding is of their sum; with few rows two
// terms, for there the matrix unit has time. The sum of the unrounded p, the
// maxima and the accumulators are fp32.
//
// Layout: no operand crosses lanes. The first product computes S^T = K Q^T,
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

namespace fq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 64;   // tokens a wave takes at once
constexpr int kRows = 16;   // query rows of a workgroup
constexpr int kMaxSplits = 1024;
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

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

// cap * tanh(x / cap), by exp: 1 - 2 / (e^{2y} + 1).
__device__ __forceinline__ float soft_cap(float x, float cap, float inv_cap)
{
    const float e = __builtin_amdgcn_exp2f(x * inv_cap * (2.0f * kLog2e));
    return cap * (1.0f - 2.0f / (e + 1.0f));
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

// Four dims of an output row from its maximum (base 2), sum and accumulator.
__device__ __forceinline__ void finish(const AttnArgs& a, int64_t rid, int dim, int d, float top, float sum, f32x4 v)
{
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        b[e] = __builtin_bit_cast(uint16_t, (__bf16)(v[e] * inv));
    *(u32x2*)(a.out + rid * dim + d) = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
    if (a.lse && d == 0)
        a.lse[rid] = sum > 0.0f ? (top + __log2f(sum)) * kLn2 : -kInf;
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
    const float sc2 = a.scale * kLog2e;
    const float inv_cap = a.softcap > 0.0f ? 1.0f / a.softcap : 0.0f;
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
        if (a.softcap > 0.0f) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] = soft_cap(x[e] * v.ks * a.scale, a.softcap, inv_cap) * kLog2e;
        } else {
            const float f = v.ks * sc2;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] *= f;
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
            if (d == 0)
                *(float2*)(a.ws + (rid * a.splits + split) * 2) = make_float2(top, sum);
            *(f32x4*)(a.ws + kv.total_q * a.q_heads * (int64_t)a.splits * 2 + (rid * a.splits + split) * D + d) = v;
        } else {
            finish(a, rid, D, d, top, sum, v);
        }
    }
}

// ---------------------------------------------------------------- many rows
// Prompts and chunks: a workgroup takes 8 waves of 16 RT query rows of one
// head group and walks over the keys in steps of 64. The step's codes are
// read once, widened to bf16 once, and shared in LDS; the next step's are
// under way meanwhile. Bound by the vector unit as much as by the matrix
// unit: 16 x 64 scores cost 32 matrix instructions (512 cycles) and, at an
// exponential and five operations each, about as many cycles of softmax, so
// two waves a SIMD alternate between the two.
//
// LDS rows: a token's dims (keys) or a dim's 64 tokens (values) in 16-byte
// chunks, turned so that reads of 16 bytes a lane meet no bank twice. The
// hardware serves 16 lanes at once, eight of one lane group with eight others
// of the next. A dim's row is half the banks: tokens 16 g + 8 k .. + 7 are chunk
// g + 4 k, at (g + 4 k) ^ (d % 8). A token's row is all of them or more (half
// with 64 dims): chunk c of token t sits at c ^ key_turn(t), which numbers the
// 16 tokens that are read together (16 (r / 4) + 4 n + r % 4 for r = 0..15).
template <int D>
__device__ __forceinline__ int key_turn(int t)
{
    return (t & 3) | (t >> 2 & (D == 64 ? 4 : 12));
}

template <int D>
struct KvStage {
    uint16_t k[kStep * D], v[D * kStep];
};

// Query rows of a workgroup: 32 a wave, 16 with 256 dims, whose accumulators
// would not fit twice.
constexpr int tile_rows(int dim) { return dim == 256 ? 128 : 256; }

template <int D, int FMT>
__global__ __launch_bounds__(512, 2) void k_attn_tile(AttnArgs a)
{
    constexpr int kTileRows = tile_rows(D), kWaveRows = kTileRows / 8, RT = kWaveRows / 16;
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

    bf16x8 q[RT][KK];
    int pos[RT], oldest[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        const int r = min(w0 + u * 16 + row, rows - 1);
        const int tok = r / group, head = h * group + r % group;
        pos[u] = s.len - s.nq + tok;
        oldest[u] = a.window > 0 ? pos[u] - a.window + 1 : -0x7fffffff;
        const uint16_t* p = a.q + (s.q0 + tok) * a.q_stride + (int64_t)head * D + grp * 8;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            // a negative scale turns the queries' signs, so that scores rise with their products
            const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
            q[u][k] = __builtin_bit_cast(bf16x8, ld16(p + k * 32) ^ u32x4{flip, flip, flip, flip});
        }
    }
    const float scale = fabsf(a.scale), sc2 = scale * kLog2e;
    const float inv_cap = a.softcap > 0.0f ? 1.0f / a.softcap : 0.0f;

    float m[RT], l[RT];
    f32x4 o[RT][T];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        m[u] = -kInf;
        l[u] = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t)
            o[u][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

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
                sw = key_turn<D>(t);
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
        f32x4 x[RT][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int t = (row >> 2) * 16 + n * 4 + (row & 3);
#pragma unroll
            for (int u = 0; u < RT; ++u)
                x[u][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KK; ++k) {
                const bf16x8 kf = *(const bf16x8*)(st.k + t * D + ((k * 4 + grp) ^ key_turn<D>(t)) * 8);
#pragma unroll
                for (int u = 0; u < RT; ++u)
                    x[u][n] = mfma(kf, q[u][k], x[u][n]);
            }
        }
        // scores stay products until the exponential: x f - m is one fused
        // operation, and with f >= 0 the largest x has the largest score
        // (f > 0 also where no token of the group is seen and its scale may be
        // anything: a hidden score is -inf times f)
        const float f = a.softcap > 0.0f ? kLog2e : fmaxf(ks * sc2, 1e-30f);
        // The row tiles go through the softmax side by side, with two branches
        // for all of them: their chains of dependent operations overlap.
        bool inside = t0 >= sp.lo && t0 + kStep <= sp.hi && ok;
#pragma unroll
        for (int u = 0; u < RT; ++u)
            inside = inside && t0 + kStep - 1 <= pos[u] && t0 >= oldest[u];
        if (a.softcap > 0.0f) {
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[u][e >> 2][e & 3] = soft_cap(x[u][e >> 2][e & 3] * ks * scale, a.softcap, inv_cap);
        }
        if (!__all(inside)) {
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int t = tv + e;
                    const bool see = ok && t >= sp.lo && t < sp.hi && t <= pos[u] && t >= oldest[u];
                    x[u][e >> 2][e & 3] = see ? x[u][e >> 2][e & 3] : -kInf;
                }
        }
        float top[RT];
        bool rises = false;
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            top[u] = x[u][0][0];
#pragma unroll
            for (int e = 1; e < 16; ++e)
                top[u] = fmaxf(top[u], x[u][e >> 2][e & 3]);
            top[u] = max_groups(top[u] == -kInf ? -kInf : top[u] * f);
            rises = rises || top[u] > m[u] + kSlack;
        }
        if (__any(rises)) {  // as in k_attn
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                const float mn = fmaxf(m[u], top[u]);
                const float alpha = __builtin_amdgcn_exp2f(m[u] - (mn == -kInf ? 0.0f : mn));
                m[u] = mn;
                l[u] *= alpha;
#pragma unroll
                for (int t = 0; t < T; ++t)
                    o[u][t] *= alpha;
            }
        }
        bf16x8 p[RT][2];
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            const float mu = m[u] == -kInf ? 0.0f : m[u];
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][e >> 2][e & 3], f, -mu));
                sum[e & 3] += y;
                p[u][e >> 3][e & 7] = (__bf16)(y * vs);
            }
            l[u] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int d = t * 16 + row;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bf16x8 vf = *(const bf16x8*)(st.v + d * kStep + ((grp + 4 * k) ^ (d & 7)) * 8);
#pragma unroll
                for (int u = 0; u < RT; ++u)
                    o[u][t] = mfma(vf, p[u][k], o[u][t]);
            }
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
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        float sum = l[u];
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        const int r = r0 + w * kWaveRows + u * 16 + row;
        if (r < rows) {
            const int64_t rid = (s.q0 + r / group) * a.q_heads + h * group + r % group;
#pragma unroll
            for (int t = 0; t < T; ++t)
                finish(a, rid, D, t * 16 + grp * 4, m[u], sum, o[u][t]);
        }
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
    const float2* ml = (const float2*)a.ws + rid * a.splits;
    const float* from = a.ws + kv.total_q * a.q_heads * (int64_t)a.splits * 2 + rid * a.splits * D;
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
        k_attn_tile<D, FMT><<<dim3((unsigned)(a.tiles * a.kv.heads), (unsigned)a.kv.batch), 512, 0, st>>>(a);
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
    const int64_t group = a.q_heads / kv.heads;
    // The kernel for many rows, where its workgroups fill the chip and their
    // rows: a step of 64 keys costs it 2.6 us for up to 256 workgroups, and the
    // kernel for few rows about 1.2 ns a tile of 16 rows. Measured at 128 dims,
    // many against few: 2 chunks of 2048 rows, 32 heads, up to 8192 keys 560 and
    // 1122 us; 8 of 128 rows 93 and 86; 1 of 2048 rows, 8 heads 87 and 36; 64 of
    // 4 rows, 32 heads over 2 171 and 59.
    const int64_t wide = tile_rows(kv.dim);
    const int64_t few_tiles = kv.batch * kv.heads * cdiv(kv.max_q * group, kRows);
    const int64_t many_tiles = kv.batch * kv.heads * cdiv(kv.max_q * group, wide);
    a.rows = kRows;
    if (cdiv(many_tiles, 256) * 2200 < few_tiles * (kv.dim == 256 ? 2 : 1)) {
        a.rows = (int)wide;
        a.tiles = (int)cdiv(kv.max_q * group, wide);
        a.chunk = kv.max_len;
        a.splits = 1;
        return 0;
    }
    a.tiles = (int)cdiv(kv.max_q * group, kRows);
    const int64_t tiles = (int64_t)kv.batch * kv.heads * a.tiles;
    int64_t span = kv.max_len;
    if (a.window > 0 && span > (int64_t)a.window + kv.max_q + kStep)
        span = (int64_t)a.window + kv.max_q + kStep;
    // One workgroup per tile if the tiles alone fill the chip, else about two
    // workgroups a CU, each with at least a step for each of its four waves
    // (4 sequences of up to 131072: 16 splits 164 us, 32 177, 64 169, 128 171;
    // 64 of up to 8192: one 119 us, two 131, eight 120). A short run of keys
    // on few tiles stays whole, on eight waves: no second launch.
    a.waves = 4;
    int64_t splits = tiles >= 512 ? 1 : cdiv(512, tiles > 0 ? tiles : 1);
    if (splits > 1 && span <= 1024 && kv.dim <= 128) {
        a.waves = 8;
        splits = 1;
    }
    if (span < 1)
        span = 1;
    splits = splits < kMaxSplits ? splits : kMaxSplits;
    const int64_t chunk = cdiv(cdiv(span, splits), 4 * kStep) * (4 * kStep);
    a.chunk = (int)chunk;
    a.splits = (int)cdiv(span, chunk);
    if (a.splits == 1)
        return 0;
    return (size_t)(kv.total_q * a.q_heads) * a.splits * (kv.dim + 2) * sizeof(float);
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
