// k_kv.hip -- writes keys and values into the paged 8-bit cache.
//
// One power-of-two scale serves a block of tokens of one head: with a =
// max|x| over the block's tokens, s = 2^p, p the smallest integer >= -126
// with a <= Fmax * 2^p, and q = Q(x / s), the division exact. A block fills
// over several calls; s only grows (s(max(a, b)) = max(s(a), s(b))), and when
// it does the codes already there move to the new scale by a power of two.
// That is exact but for results in the format's subnormals, so what a block
// holds does not depend on how its tokens were split over calls, but for
// those.
//
// Bound by latency for single tokens (lengths, then page and rows, then the
// codes) and by memory for prompts. One workgroup takes one block of one head
// (several where sequences are very unequal), K or V, and holds its rows in
// registers between the amax and the cast (a block of up to 8 16-byte loads a
// thread: 64 tokens of 128 bf16 dims take 4; larger ones are read again, from
// cache). The cache holds V transposed (k_attn.hip says why): a thread takes
// four tokens of the same dims, and the converter packs them token by token, so
// the transposed code words come out of registers with no exchange.
#include "codec.hpp"
#include "launch.hpp"

namespace fq {
namespace {

// Exponent p of the block scale: a = 1.M * 2^(E - 127), Fmax = 1.75 * 2^kEmax.
template <int FMT>
__device__ __forceinline__ int scale_exp(float a)
{
    const uint32_t b = __float_as_uint(a) & 0x7fffffffu;
    const int p = (int)(b >> 23) - 127 - Fmt<FMT>::kEmax + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(p, -126);  // at most 121, which an infinity or a NaN gives
}

template <int FMT>
__device__ __forceinline__ float dec1(uint32_t code)
{
    return FMT == kE4M3 ? dec_e4m3(code) : dec_e5m2(code);
}

// Codes c moved to another scale, r the ratio of the old to the new one.
template <int FMT>
__device__ __forceinline__ uint32_t move4(uint32_t c, float r)
{
    return enc4<FMT>(dec1<FMT>(c & 0xffu), dec1<FMT>(c >> 8 & 0xffu), dec1<FMT>(c >> 16 & 0xffu), dec1<FMT>(c >> 24), r);
}

constexpr int kHold = 8;

// The block of tokens [base, base + kv.block) of sequence `seq`, the first new
// token of which is at position `first`.
template <typename T, int FMT, bool IS_V>
__device__ __forceinline__ void append_block(const KvArgs& kv, const T* fresh, int64_t stride, int seq, int h,
                                             const KvSeq& s, int first, int base, int tid, float* red)
{
    constexpr int E = In<T>::kE;
    const int lo = max(base, first), hi = min(base + kv.block, s.len);  // (base is not negative)
    const int page = kv.table[(int64_t)seq * kv.max_pages + base / kv.page];
    const int dim = kv.dim, in_page = base & (kv.page - 1);
    const int at = lo - base, cnt = hi - lo;  // the new tokens of the block
    const int per_row = dim / E, shift = 31 - __clz(per_row);
    const T* x = fresh + (s.q0 + lo - first) * stride + (int64_t)h * dim;

    // Load j of this thread. K: 16 bytes of a token, consecutive threads along
    // the token. V: token j % 4 of a group of four, dims dim_of(j); the groups
    // run fastest.
    const int g0 = at >> 2, groups = ((at + cnt - 1) >> 2) - g0 + 1;
    const int total = IS_V ? groups * per_row * 4 : cnt * per_row;   // loads of the block
    const int loads = IS_V ? (int)cdiv(groups * per_row, kWG) * 4 : (int)cdiv(total, kWG);
    auto place = [&](int j, int& tok, int& d) {  // token of the block and first dim; false: none
        if constexpr (IS_V) {
            const int u = tid + (j >> 2) * kWG, c = u / groups;
            tok = (g0 + u - c * groups) * 4 + (j & 3);
            d = c * E;
            return c < per_row && tok >= at && tok < at + cnt;
        } else {
            const int i = tid + j * kWG;
            tok = at + (i >> shift);
            d = (i & (per_row - 1)) * E;
            return i < total;
        }
    };
    auto load = [&](int j) {
        int tok, d;
        return place(j, tok, d) ? ld16(x + (int64_t)(tok - at) * stride + d) : u32x4{0u, 0u, 0u, 0u};
    };
    u32x4 hold[kHold];
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        hold[j] = j < loads ? load(j) : u32x4{0u, 0u, 0u, 0u};
    if (page < 0 || page >= kv.num_pages)
        return;
    const int64_t tile = ((int64_t)page * kv.heads + h) * kv.page;  // in tokens
    float* scale = (IS_V ? kv.vs : kv.ks) + (tile + in_page) / kv.block;
    uint8_t* codes = (IS_V ? kv.v : kv.k) + tile * dim;
    const float olds = at > 0 ? *scale : 0.0f;
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        a = fmaxf(a, In<T>::absmax16(hold[j]));
    for (int j = kHold; j < loads; ++j)
        a = fmaxf(a, In<T>::absmax16(load(j)));
    a = max_workgroup(a, red);  // (every thread has read the old scale)
    const int p = scale_exp<FMT>(a);
    const float mine = __uint_as_float((uint32_t)(p + 127) << 23);
    const bool grows = at > 0 && mine > olds;
    const float sc = at > 0 && !grows ? olds : mine;
    if (tid == 0)
        *scale = sc;
    // x / s as a product where s is a power of two, and a quotient where an older
    // scale that is none stands: x times a rounded inverse misses ties
    const bool whole = (__float_as_uint(sc) & 0x7fffffu) == 0;
    const float inv = sc == mine ? __uint_as_float((uint32_t)(127 - p) << 23) : whole ? 1.0f / sc : 1.0f;
    auto unpack = [&](u32x4 v, float* f) {
        In<T>::unpack(v, f);
        if (!whole) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                f[e] /= sc;
        }
    };

    if (grows) {  // the block's older tokens, [0, at), move to the new scale
        const float r = olds * inv;
        // 16 codes a thread, two loads under way: K's tokens are one run, V's
        // are runs of 16 in each dim's row, and a rest of less than 16
        const int runs = IS_V ? at >> 4 : at * (dim >> 4);
        const int n = IS_V ? runs * dim : runs;
        auto place16 = [&](int i) {
            if constexpr (!IS_V)
                return codes + (int64_t)in_page * dim + i * 16;
            const int d = i / runs;
            return codes + (int64_t)d * kv.page + in_page + (i - d * runs) * 16;
        };
        auto move16 = [&](u32x4 c) {
            return u32x4{move4<FMT>(c[0], r), move4<FMT>(c[1], r), move4<FMT>(c[2], r), move4<FMT>(c[3], r)};
        };
        for (int i = tid; i < n; i += 2 * kWG) {
            const bool two = i + kWG < n;
            uint8_t* c0 = place16(i);
            uint8_t* c1 = two ? place16(i + kWG) : c0;
            const u32x4 v0 = ld16(c0), v1 = ld16(c1);
            *(u32x4*)c0 = move16(v0);
            if (two)
                *(u32x4*)c1 = move16(v1);
        }
        if (IS_V && (at & 15)) {
            // whole words of four tokens, and by bytes the word that new tokens share
            const int from = at & ~15, words = (at - from + 3) >> 2;
            for (int i = tid; i < dim * words; i += kWG) {
                const int d = i / words, t = from + (i - d * words) * 4;
                uint8_t* c = codes + (int64_t)d * kv.page + in_page + t;
                if (t + 4 <= at) {
                    *(uint32_t*)c = move4<FMT>(*(uint32_t*)c, r);
                } else {
                    for (int b = 0; b < at - t; ++b)
                        c[b] = enc1<FMT>(dec1<FMT>(c[b]), r);
                }
            }
        }
    }
    if constexpr (!IS_V) {
        auto put = [&](int j, u32x4 v) {
            int tok, d;
            if (!place(j, tok, d))
                return;
            float f[E];
            unpack(v, f);
            uint32_t* o = (uint32_t*)(codes + (int64_t)(in_page + tok) * dim + d);
            if constexpr (E == 8)
                *(u32x2*)o = u32x2{enc4<FMT>(f[0], f[1], f[2], f[3], inv), enc4<FMT>(f[4], f[5], f[6], f[7], inv)};
            else
                *o = enc4<FMT>(f[0], f[1], f[2], f[3], inv);
        };
#pragma unroll
        for (int j = 0; j < kHold; ++j)
            if (j < loads)
                put(j, hold[j]);
        for (int j = kHold; j < loads; ++j)
            put(j, load(j));
    } else {
        auto put = [&](int j, u32x4 v0, u32x4 v1, u32x4 v2, u32x4 v3) {
            const int u = tid + (j >> 2) * kWG, c = u / groups;
            if (c >= per_row)
                return;
            const int t = (g0 + u - c * groups) * 4;
            const int from = max(at - t, 0), to = min(at + cnt - t, 4);
            float f0[E], f1[E], f2[E], f3[E];
            unpack(v0, f0);
            unpack(v1, f1);
            unpack(v2, f2);
            unpack(v3, f3);
            uint8_t* o = codes + (int64_t)(c * E) * kv.page + in_page + t;
#pragma unroll
            for (int e = 0; e < E; ++e, o += kv.page) {
                const uint32_t q = enc4<FMT>(f0[e], f1[e], f2[e], f3[e], inv);
                if (from == 0 && to == 4) {
                    *(uint32_t*)o = q;
                } else {
                    for (int b = from; b < to; ++b)
                        o[b] = (uint8_t)(q >> (8 * b));
                }
            }
        };
#pragma unroll
        for (int j = 0; j < kHold; j += 4)
            if (j < loads)
                put(j, hold[j], hold[j + 1], hold[j + 2], hold[j + 3]);
        for (int j = kHold; j < loads; j += 4)
            put(j, load(j), load(j + 1), load(j + 2), load(j + 3));
    }
}

template <typename T, int FMT>
__global__ __launch_bounds__(kWG) void k_kv_append(KvArgs kv, const T* knew, int64_t kstride, const T* vnew,
                                                   int64_t vstride)
{
    __shared__ float red[4];
    const int seq = (int)blockIdx.y, is_v = (int)blockIdx.z >= kv.heads, h = (int)blockIdx.z - is_v * kv.heads;
    const KvSeq s = kv_seq(kv, seq);
    const int first = s.len - s.nq;  // position of the first new token (below 0: it is not stored)
    const int start = max(first, 0);
    if (start >= s.len)
        return;
    for (int base = start / kv.block * kv.block + (int)blockIdx.x * kv.block; base < s.len;
         base += (int)gridDim.x * kv.block) {
        // read anew in every turn: what follows from it would otherwise be kept
        // over the loop, in 127 registers instead of 73
        int tid = (int)threadIdx.x;
        asm volatile("" : "+v"(tid));
        if (is_v)
            append_block<T, FMT, true>(kv, vnew, vstride, seq, h, s, first, base, tid, red);
        else
            append_block<T, FMT, false>(kv, knew, kstride, seq, h, s, first, base, tid, red);
    }
}

// Workgroups of a sequence and head: one for each block that max_q tokens can
// touch, unless the sequences are of such different lengths that most of them
// would find nothing. They are held to four times what total_q rows of equal
// sequences would need, and take several blocks each.
template <typename T, int FMT>
hipError_t append(const KvArgs& kv, const void* k, int64_t ks, const void* v, int64_t vs, hipStream_t st)
{
    const int64_t per = (kv.max_q + kv.block - 2) / kv.block + 1;
    const int64_t most = cdiv(4 * (cdiv(kv.total_q, kv.block) + 2 * (int64_t)kv.batch), kv.batch);
    const dim3 grid((unsigned)(per < most ? per : most), (unsigned)kv.batch, (unsigned)kv.heads * 2);
    k_kv_append<T, FMT><<<grid, kWG, 0, st>>>(kv, (const T*)k, ks, (const T*)v, vs);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvArgs& kv, int bf, const void* k, int64_t ks, const void* v, int64_t vs,
                            hipStream_t st)
{
    if (kv.fmt == kE4M3)
        return bf ? append<uint16_t, kE4M3>(kv, k, ks, v, vs, st) : append<float, kE4M3>(kv, k, ks, v, vs, st);
    return bf ? append<uint16_t, kE5M2>(kv, k, ks, v, vs, st) : append<float, kE5M2>(kv, k, ks, v, vs, st);
}

}  // namespace fq
