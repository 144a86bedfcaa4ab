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
// Bound by launch latency for single tokens and by memory for prompts: the
// new rows are read twice (amax, cast), the second time from cache. One
// workgroup takes one block of one head, K or V; V's codes turn in LDS,
// because the cache holds V transposed (k_attn.hip says why).
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

constexpr int kMaxBlock = 128, kMaxDim = 256;

template <typename T, int FMT>
__global__ __launch_bounds__(kWG) void k_kv_append(KvArgs kv, const T* knew, int64_t kstride, const T* vnew,
                                                   int64_t vstride, int blocks_per_seq)
{
    __shared__ float red[4];
    __shared__ uint8_t turn[kMaxDim * (kMaxBlock + 4)];
    const int seq = (int)(blockIdx.x / (unsigned)blocks_per_seq);
    const int nth = (int)blockIdx.x - seq * blocks_per_seq;
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const KvSeq s = kv_seq(kv, seq);
    const int first = s.len - s.nq;  // position of the first new token (below 0: it is not stored)
    const int start = max(first, 0);
    const int base = (start / kv.block + nth) * kv.block;
    const int lo = max(base, start), hi = min(base + kv.block, s.len);
    if (lo >= hi)
        return;
    const int page = kv.table[(int64_t)seq * kv.max_pages + base / kv.page];
    if (page < 0 || page >= kv.num_pages)
        return;
    const int dim = kv.dim, in_page = base & (kv.page - 1);
    const int64_t tile = ((int64_t)page * kv.heads + h) * kv.page;  // in tokens
    float* scale = (is_v ? kv.vs : kv.ks) + (tile + in_page) / kv.block;
    uint8_t* codes = (is_v ? kv.v : kv.k) + tile * dim;
    const int64_t stride = is_v ? vstride : kstride;
    const T* x = (is_v ? vnew : knew) + (s.q0 + lo - first) * stride + (int64_t)h * dim;
    constexpr int E = In<T>::kE;
    const int per_row = dim / E, n = (hi - lo) * per_row;
    const int shift = 31 - __clz(per_row);

    float a = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kWG)
        a = fmaxf(a, In<T>::absmax16(ld16(x + (i >> shift) * stride + (i & (per_row - 1)) * E)));
    const float olds = lo > base ? *scale : 0.0f;
    a = max_workgroup(a, red);
    const int p = scale_exp<FMT>(a);
    const float mine = __uint_as_float((uint32_t)(p + 127) << 23);
    const bool grows = lo > base && mine > olds;
    const float sc = lo > base && !grows ? olds : mine;
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0)
        *scale = sc;
    // x / s: s is 2^p unless an older, larger scale stands
    const float inv = sc == mine ? __uint_as_float((uint32_t)(127 - p) << 23) : 1.0f / sc;

    if (grows) {  // the block's older tokens move to the new scale
        const float r = olds * inv;
        const int old = lo - base;
        for (int i = threadIdx.x; i < old * dim; i += kWG) {
            uint8_t* c = is_v ? codes + (int64_t)(i / old) * kv.page + in_page + i % old : codes + (int64_t)in_page * dim + i;
            *c = enc1<FMT>(dec1<FMT>(*c), r);
        }
    }
    if (!is_v) {
        uint8_t* q = codes + (int64_t)(in_page + lo - base) * dim;
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kWG) {
            float f[E];
            In<T>::unpack(ld16(x + (i >> shift) * stride + (i & (per_row - 1)) * E), f);
            uint32_t* o = (uint32_t*)(q + (int64_t)i * E);
#pragma unroll
            for (int e = 0; e < E; e += 4)
                o[e / 4] = enc4<FMT>(f[e], f[e + 1], f[e + 2], f[e + 3], inv);
        }
        return;
    }
    const int at = lo - base, cnt = hi - lo, pitch = kv.block + 4;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kWG) {
        float f[E];
        const int t = i >> shift, d = (i & (per_row - 1)) * E;
        In<T>::unpack(ld16(x + t * stride + d), f);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const uint32_t w = enc4<FMT>(f[e], f[e + 1], f[e + 2], f[e + 3], inv);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                turn[(d + e + b) * pitch + at + t] = (uint8_t)(w >> (8 * b));
        }
    }
    __syncthreads();
    uint8_t* q = codes + in_page;
    if (cnt == kv.block) {
        const int quads = kv.block >> 2, qs = 31 - __clz(quads);
        for (int i = threadIdx.x; i < dim * quads; i += kWG) {
            const int d = i >> qs, c = (i & (quads - 1)) * 4;
            *(uint32_t*)(q + (int64_t)d * kv.page + c) = *(const uint32_t*)(turn + d * pitch + c);
        }
        return;
    }
    for (int i = threadIdx.x; i < dim * cnt; i += kWG) {
        const int d = i / cnt, c = at + i % cnt;
        q[(int64_t)d * kv.page + c] = turn[d * pitch + c];
    }
}

template <typename T, int FMT>
hipError_t append(const KvArgs& kv, const void* k, int64_t ks, const void* v, int64_t vs, hipStream_t st)
{
    const int per = (kv.max_q + kv.block - 2) / kv.block + 1;  // blocks that max_q tokens can touch
    const dim3 grid((unsigned)((int64_t)kv.batch * per), (unsigned)kv.heads, 2);
    k_kv_append<T, FMT><<<grid, kWG, 0, st>>>(kv, (const T*)k, ks, (const T*)v, vs, per);
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
