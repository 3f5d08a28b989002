// k_rope_rows.cu - rotary positions of packed rows of queries and keys.
//
// Row t of q [T, H, dh] and k [T, Hkv, dh] has position p = positions[t]; the pair
// (a, b) number i of every head's first `rot` coordinates becomes
//   (a cos - b sin, a sin + b cos) mscale,  angle = p inv_freq[i],
// pairs being (x[2i], x[2i+1]) or (x[i], x[i + rot/2]); coordinates from rot on are
// copied.  Everything is fp32 after the angle, rounded once.
//
// The angle: positions reach 2^31 and the angle counts modulo one turn, so the turns per
// position are held as a 64-bit fraction (inv_freq / 2 pi modulo 1).  Its product with the
// position in 64-bit integers wraps by itself, exactly, to the fraction of a turn; fp32 takes
// over from there (sincospi).  The fraction is made of inv_freq's mantissa by integer
// products as well: GB300 has two fp64 lanes a clock and SM, and one fp64 product per thread and
// pair would take longer than the rows.
//
// Bound by memory: each row is read and written once, 16 bytes per lane and access; 8 or 4 where rows,
// strides or halves of pairs begin on no more (22041 tokens of 3/3 x 80, 40 turned in halves: 17.8 us,
// element by element 68).  A warp takes a
// token (where they are few, some of its heads): it asks for its first rows, computes the token's
// sines into 1 KB of shared memory of its own meanwhile, and turns row after row (32768 tokens of 16/4 x 128: 58 us,
// 0.87 of a copy's bandwidth).  No barrier: with the sines of 16 tokens shared by a CTA, sines and
// rows took turns (62 to 72 us), and with sines in registers, a thread for one vector of all
// heads, too few bytes were on their way (85 us).
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 6;                         // of an SM (k_rope_rows; 4 with two rows on their way: 61 us; 8: 73)
constexpr int kRopeTokens = 16;                     // at most, per round of a CTA

struct RopeGeom {
    int T, H, Hkv, dh, rot;
    int tokens;                                      // per round
    int heads_per;                                   // of a CTA (grid.y) or warp, heads of q and k together
    int cols, pair_cols;                             // k_rope_rows: vectors of a head (partners count once); with pairs
    int lanes;                                       // k_rope_rows: lanes of a row, a power of two
    int splits;                                      // k_rope_rows: warps of a token
    int copy_tail;                                   // coordinates behind rot are copied
    float mscale;
    int64_t s[8];                                    // q, k, q_out, k_out: token, head strides
};

template <typename T>
__device__ __forceinline__ float as_f32(T v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
    if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
    else return v;
}

// inv_freq / (2 pi) modulo 1, times 2^64: the mantissa times 2^66 / (2 pi), shifted by the exponent.
__device__ __forceinline__ unsigned long long turns_of(double inv_freq) {
    const long long bits = __double_as_longlong(inv_freq);
    const int e = (int)(bits >> 52) & 2047;
    const unsigned long long man = ((unsigned long long)bits << 11) | 0x8000000000000000ull;
    unsigned long long t = __umul64hi(man, 0xA2F9836E4E441529ull);     // inv_freq / (2 pi) = t 2^(e - 1088)
    const int up = e - 1024;
    t = up >= 64 || up <= -64 ? 0 : up >= 0 ? t << up : t >> -up;
    return bits < 0 ? 0ull - t : t;
}
__device__ __forceinline__ float2 cos_sin(unsigned long long turns, int position, float mscale) {
    const long long w = (long long)(turns * (unsigned long long)(long long)position);
    float sn, cn;
    sincospif((float)w * 0x1p-63f, &sn, &cn);                          // 2 x the fraction of a turn
    return make_float2(cn * mscale, sn * mscale);
}

template <typename T, int VE>
struct __align__(VE * sizeof(T)) Elems {
    T v[VE];
};

// Rows are read past the L1 cache, as in k_cache8.cu: a launch that overlaps the end of the one before may share an SM with
// its reads of lines that other SMs went on to write (rows of 40 bytes, say, turned in place).
template <typename V>
__device__ __forceinline__ V past_l1(const V* p) {
    using R = std::conditional_t<sizeof(V) == 16, uint4, std::conditional_t<sizeof(V) == 8, uint2,
              std::conditional_t<sizeof(V) == 4, unsigned, unsigned short>>>;
    const R r = __ldcg(reinterpret_cast<const R*>(p));
    V v;
    memcpy(&v, &r, sizeof v);
    return v;
}

template <typename T>
__device__ __forceinline__ void turn_pair(T& x, T& y, float2 r) {
    const float a = as_f32(x), b = as_f32(y);
    x = from_f32<T>(a * r.x - b * r.y);
    y = from_f32<T>(a * r.y + b * r.x);
}

// The sines of nt tokens from t0 on.
__device__ __forceinline__ void fill_sines(float2* cs, unsigned long long turns, const int32_t* __restrict__ positions, int t0,
                                           int nt, int half, float mscale) {
    const int pair = threadIdx.x % half, first = threadIdx.x / half, step = kRopeThreads / half;
    if (first < step)
        for (int t = first; t < nt; t += step) cs[t * half + pair] = cos_sin(turns, positions[t0 + t], mscale);
}

// Accesses of VB bytes: every pointer and stride a multiple of them, the pairs of a vector whole.
template <typename T, bool INTER, int VB>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    k_rope_rows(const T* q, const T* k, T* qo, T* ko,                  // outputs may be the inputs
                const int32_t* __restrict__ positions, const double* __restrict__ inv_freq, const RopeGeom g) {
    constexpr int VE = VB / (int)sizeof(T);
    constexpr int NP = INTER ? VE / 2 : VE;                            // pairs of a vector
    using Vec = Elems<T, VE>;
    __shared__ unsigned long long turns[128];
    __shared__ __align__(16) float2 sines[kRopeThreads / 32][128];
    const int half = g.rot >> 1, tid = threadIdx.x, lane = tid & 31;
    float2* cs = sines[tid >> 5];
    pdl_wait();
    pdl_trigger();
    if (tid < half) turns[tid] = turns_of(inv_freq[tid]);
    __syncthreads();
    const int x0 = lane & (g.lanes - 1), row = lane / g.lanes, rows = 32 / g.lanes;
    const int warps = (int)gridDim.x * (kRopeThreads / 32);
    const int items = g.T * g.splits;
    for (int item = (int)blockIdx.x * (kRopeThreads / 32) + (tid >> 5); item < items; item += warps) {
        const int t = g.splits == 1 ? item : item / g.splits;
        const int h0 = (item - t * g.splits) * g.heads_per, h1 = min(h0 + g.heads_per, g.H + g.Hkv);
        const int p = __ldg(positions + t);
        bool sined = false;
        for (int x = x0; x < g.cols || !sined; x += 32) {              // (more than 32 columns: fp32 heads of 256)
            const bool pairs = x < g.pair_cols;
            const int e = pairs ? x * VE : g.rot + (x - g.pair_cols) * VE;     // a column without pairs is copied
            for (int h = h0 + row; h < h1 || !sined; h += rows) {
                const bool live = h < h1 && x < g.cols, isq = h < g.H;
                const int hh = isq ? h : h - g.H;
                Vec lo, hi;
                if (live) {
                    const T* src = (isq ? q : k) + (int64_t)t * g.s[isq ? 0 : 2] + (int64_t)hh * g.s[isq ? 1 : 3] + e;
                    lo = past_l1(reinterpret_cast<const Vec*>(src));
                    if (!INTER && pairs) hi = past_l1(reinterpret_cast<const Vec*>(src + half));
                }
                if (!sined) {                                          // the whole warp, once a token
                    sined = true;
                    __syncwarp();
                    for (int j = lane; j < half; j += 32) cs[j] = cos_sin(turns[j], p, g.mscale);
                    __syncwarp();
                }
                if (!live) continue;
                T* dst = (isq ? qo : ko) + (int64_t)t * g.s[isq ? 4 : 6] + (int64_t)hh * g.s[isq ? 5 : 7] + e;
                if (pairs) {
                    const float4* r4 = reinterpret_cast<const float4*>(cs + (INTER ? x * NP : e));
                    if constexpr (NP == 1) turn_pair(lo.v[0], lo.v[1], cs[x]);
#pragma unroll
                    for (int j = 0; j + 1 < NP; j += 2) {
                        const float4 r = r4[j >> 1];
                        if constexpr (INTER) {
                            turn_pair(lo.v[2 * j], lo.v[2 * j + 1], make_float2(r.x, r.y));
                            turn_pair(lo.v[2 * j + 2], lo.v[2 * j + 3], make_float2(r.z, r.w));
                        } else {
                            turn_pair(lo.v[j], hi.v[j], make_float2(r.x, r.y));
                            turn_pair(lo.v[j + 1], hi.v[j + 1], make_float2(r.z, r.w));
                        }
                    }
                    if constexpr (!INTER) *reinterpret_cast<Vec*>(dst + half) = hi;
                }
                *reinterpret_cast<Vec*>(dst) = lo;
            }
        }
    }
}

// Halves of an odd number of bf16 elements and the like, element by element: the sines of a few tokens in shared memory for all heads.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
    k_rope_plain(const T* q, const T* k, T* qo, T* ko, const int32_t* __restrict__ positions,
                 const double* __restrict__ inv_freq, const RopeGeom g) {
    __shared__ float2 cs[kRopeTokens * 128];
    const int half = g.rot >> 1, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const unsigned long long turns = turns_of(inv_freq[tid % half]);
    const int h0 = (int)blockIdx.y * g.heads_per, heads = min(g.heads_per, g.H + g.Hkv - h0);
    const int per = half + (g.copy_tail ? g.dh - g.rot : 0);             // pairs of a head, then the copied tail
    const int chunks = (g.T + g.tokens - 1) / g.tokens;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t0 = c * g.tokens, nt = min(g.tokens, g.T - t0);
        fill_sines(cs, turns, positions, t0, nt, half, g.mscale);
        __syncthreads();
        const int items = nt * heads * per;
        for (int i = tid; i < items; i += kRopeThreads) {
            const int x = i % per, th = i / per;
            const int h = h0 + th % heads, t = th / heads;
            const bool isq = h < g.H;
            const int hh = isq ? h : h - g.H;
            const T* src = (isq ? q : k) + (int64_t)(t0 + t) * g.s[isq ? 0 : 2] + (int64_t)hh * g.s[isq ? 1 : 3];
            T* dst = (isq ? qo : ko) + (int64_t)(t0 + t) * g.s[isq ? 4 : 6] + (int64_t)hh * g.s[isq ? 5 : 7];
            if (x >= half) {
                dst[x + half] = past_l1(src + x + half);
            } else {
                const int a = INTER ? 2 * x : x, b = INTER ? 2 * x + 1 : x + half;
                T va = past_l1(src + a), vb = past_l1(src + b);
                turn_pair(va, vb, cs[t * half + x]);
                dst[a] = va;
                dst[b] = vb;
            }
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_t(const RopeRowsArgs& a, cudaStream_t st) {
    RopeGeom g{};
    g.T = a.T;
    g.H = a.H;
    g.Hkv = a.Hkv;
    g.dh = a.dh;
    g.rot = a.rot;
    g.mscale = a.mscale;
    // bytes of an access: what every pointer, stride and part of a head is a multiple of
    const int es = sizeof(T);
    int64_t whole = 16 | (int64_t)a.dh * es | (int64_t)(a.interleaved ? a.rot : a.rot / 2) * es;
    const void* ptr[4] = {a.q, a.k, a.qo, a.ko};
    for (int i = 0; i < 8; ++i) {
        g.s[i] = a.strides[i];
        if ((i / 2) % 2 && !a.Hkv) continue;
        whole |= a.strides[i] * es | (int64_t)reinterpret_cast<uintptr_t>(ptr[i / 2]);
    }
    const int vb = (int)(whole & -whole);
    g.copy_tail = a.rot < a.dh && (a.q != a.qo || (a.Hkv && a.k != a.ko));
    const int heads = a.H + a.Hkv;
    const auto go = [&](auto kernel, dim3 grid, int smem) {
        return launch_pdl(kernel, grid, dim3(kRopeThreads), smem, st, static_cast<const T*>(a.q),
                          static_cast<const T*>(a.k), static_cast<T*>(a.qo), static_cast<T*>(a.ko), a.positions,
                          a.inv_freq, g);
    };
    if (vb > es) {
        const int ve = vb / es;
        g.pair_cols = a.interleaved ? a.rot / ve : a.rot / 2 / ve;
        g.cols = g.pair_cols + (g.copy_tail ? (a.dh - a.rot) / ve : 0);
        g.lanes = 1;
        while (g.lanes < g.cols && g.lanes < 32) g.lanes <<= 1;
        // a warp for a token; for some of its heads where the tokens are few (as many rows as its lanes take at once)
        const int least = 32 / g.lanes, most = (heads + least - 1) / least, warps = sm_count() * 16;
        g.splits = a.T >= warps / 2 ? 1 : (warps / 2 + a.T - 1) / a.T;
        if (g.splits > most) g.splits = most;
        g.heads_per = (heads + g.splits - 1) / g.splits;
        g.splits = (heads + g.heads_per - 1) / g.heads_per;
        const int64_t ctas = ((int64_t)a.T * g.splits + kRopeThreads / 32 - 1) / (kRopeThreads / 32), cap = (int64_t)sm_count() * kRopeCtas;
        const dim3 grid((unsigned)(ctas < cap ? ctas : cap));
        // A grid that could be even but leaves places free piles up on the SMs that the launch before frees first.  Shared
        // memory that nothing uses holds it to what every SM has to take: 6007 tokens of 12/12 x 64 14.3 -> 13.1 us,
        // 4000 of 16/4 x 128 13.7 -> 12.4.  (Three CTAs and fewer take 5 us or less either way.)
        constexpr int kStatic = 128 * 8 + kRopeThreads / 32 * 128 * 8;
        const int per = (int)((grid.x + sm_count() - 1) / sm_count());
        int smem = per < kRopeCtas ? 228 * 1024 / (per + 1) - kStatic : 0;
        if (kStatic + smem > 48 * 1024) smem = 0;
        if (vb == 16) return a.interleaved ? go(k_rope_rows<T, true, 16>, grid, smem) : go(k_rope_rows<T, false, 16>, grid, smem);
        if (vb == 8) return a.interleaved ? go(k_rope_rows<T, true, 8>, grid, smem) : go(k_rope_rows<T, false, 8>, grid, smem);
        if constexpr (sizeof(T) == 2)
            return a.interleaved ? go(k_rope_rows<T, true, 4>, grid, smem) : go(k_rope_rows<T, false, 4>, grid, smem);
    }
    // As many tokens a round as leave every SM a few CTAs; a step of few tokens is split
    // over the heads, each CTA with its own sines.
    const int want = sm_count() * 4;
    g.tokens = kRopeTokens;
    while (g.tokens > 1 && (a.T + g.tokens - 1) / g.tokens < want) g.tokens >>= 1;
    const int chunks = (a.T + g.tokens - 1) / g.tokens;
    int splits = chunks >= want / 2 ? 1 : (want / 2 + chunks - 1) / chunks;
    if (splits > heads) splits = heads;
    g.heads_per = (heads + splits - 1) / splits;
    splits = (heads + g.heads_per - 1) / g.heads_per;
    const int cap = sm_count() * 8, rounds = (chunks + cap - 1) / cap;
    const dim3 grid((chunks + rounds - 1) / rounds, splits);
    return a.interleaved ? go(k_rope_plain<T, true>, grid, 0) : go(k_rope_plain<T, false>, grid, 0);
}

}  // namespace

cudaError_t launch_rope_rows(const RopeRowsArgs& a, cudaStream_t st) {
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace tfm
