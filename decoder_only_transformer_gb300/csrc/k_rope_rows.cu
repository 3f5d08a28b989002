// k_rope_rows.cu - rotary positions of packed rows of queries and keys.
//
// Row t of q [T, H, dh] and k [T, Hkv, dh] has position p = positions[t]; the pair
// (a, b) number i of every head's first `rot` coordinates becomes
//   (a cos - b sin, a sin + b cos) mscale,  angle = p inv_freq[i],
// pairs being (x[2i], x[2i+1]) or (x[i], x[i + rot/2]); coordinates from rot on are
// copied.  Everything is fp32 after the angle, rounded once.
//
// The angle: positions reach 2^31 and the angle counts modulo one turn, so the turns per
// position are held as a 64-bit fraction (inv_freq / 2 pi, from fp64, modulo 1).  Its
// product with the position in 64-bit integers wraps by itself, exactly, to the fraction
// of a turn; fp32 takes over from there (sincospi).  One fp64 conversion per thread and
// call: GB300 has two fp64 lanes a clock and SM, and a sine per (token, pair) in fp64
// would cost more than the rows.
//
// Bound by memory: each row is read and written once, 16 bytes per thread and access; the
// sines of a few tokens are computed once per CTA, in shared memory, for all heads.
#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 16;                     // at most, per round of a CTA

struct RopeGeom {
    int T, H, Hkv, dh, rot;
    int tokens;                                      // per round
    int head_splits, heads_per;                      // grid.y: heads of q and k together
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

// VE consecutive elements, one 16-byte access if VE is more than one.
template <typename T, int VE>
struct __align__(VE > 1 ? 16 : sizeof(T)) Elems {
    T v[VE];
};

// VEC: 16-byte accesses (every pointer and stride a multiple of 16 bytes, and the pairs of
// a vector whole); otherwise element by element.
template <typename T, bool VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
    k_rope_rows(const T* q, const T* k, T* qo, T* ko,                  // outputs may be the inputs
                const int32_t* __restrict__ positions, const double* __restrict__ inv_freq, const RopeGeom g) {
    constexpr int VE = VEC ? 16 / (int)sizeof(T) : (INTER ? 2 : 1);      // elements of an item's vector
    using Vec = Elems<T, VEC ? VE : 1>;
    __shared__ float2 cs[kRopeTokens * 128];
    const int half = g.rot >> 1;
    const int tid = threadIdx.x;
    const int pair = tid % half, lane_tok = tid / half, toks = kRopeThreads / half;
    pdl_wait();
    pdl_trigger();
    unsigned long long turn = 0;
    if (lane_tok < toks) {
        double f = inv_freq[pair] * 0.15915494309189533576888;           // 1 / (2 pi)
        f -= floor(f);
        turn = __double2ull_rd(f * 18446744073709551616.0);
    }
    const int h0 = (int)blockIdx.y * g.heads_per, h1 = min(h0 + g.heads_per, g.H + g.Hkv);
    // items of a head: vectors with their pairs inside (INTER) or with a partner half a
    // head further; then the copied tail
    const int pv = INTER ? g.rot / VE : half / VE;
    const int tail = g.copy_tail ? (g.dh - g.rot + VE - 1) / VE : 0;     // VE = 2 element by element: odd tails too
    const int per = pv + tail;
    const int chunks = (g.T + g.tokens - 1) / g.tokens;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t0 = c * g.tokens, nt = min(g.tokens, g.T - t0);
        if (lane_tok < toks)
            for (int t = lane_tok; t < nt; t += toks) {
                const long long w = (long long)(turn * (unsigned long long)(long long)positions[t0 + t]);
                float sn, cn;
                sincospif((float)w * 0x1p-63f, &sn, &cn);                // 2 x the fraction of a turn
                cs[t * half + pair] = make_float2(cn * g.mscale, sn * g.mscale);
            }
        __syncthreads();
        const int items = nt * (h1 - h0) * per;
        for (int i = tid; i < items; i += kRopeThreads) {
            const int x = i % per, th = i / per;
            const int h = h0 + th % (h1 - h0), t = th / (h1 - h0);
            const bool isq = h < g.H;
            const int hh = isq ? h : h - g.H;
            const T* src = (isq ? q : k) + (int64_t)(t0 + t) * g.s[isq ? 0 : 2] + (int64_t)hh * g.s[isq ? 1 : 3];
            T* dst = (isq ? qo : ko) + (int64_t)(t0 + t) * g.s[isq ? 4 : 6] + (int64_t)hh * g.s[isq ? 5 : 7];
            const float2* a = cs + t * half;
            if (x >= pv) {
                const int e = g.rot + (x - pv) * VE;
                if constexpr (VEC) {
                    *reinterpret_cast<Vec*>(dst + e) = *reinterpret_cast<const Vec*>(src + e);
                } else {
                    for (int j = e; j < min(e + VE, g.dh); ++j) dst[j] = src[j];
                }
            } else if constexpr (INTER) {
                const int e = x * VE;
                T v[VE];
                if constexpr (VEC) *reinterpret_cast<Vec*>(v) = *reinterpret_cast<const Vec*>(src + e);
                else v[0] = src[e], v[1] = src[e + 1];
#pragma unroll
                for (int j = 0; j < VE; j += 2) {
                    const float2 r = a[(e + j) >> 1];
                    const float p = as_f32(v[j]), s = as_f32(v[j + 1]);
                    v[j] = from_f32<T>(p * r.x - s * r.y);
                    v[j + 1] = from_f32<T>(p * r.y + s * r.x);
                }
                if constexpr (VEC) *reinterpret_cast<Vec*>(dst + e) = *reinterpret_cast<const Vec*>(v);
                else dst[e] = v[0], dst[e + 1] = v[1];
            } else {
                const int e = x * VE;
                Vec lo = *reinterpret_cast<const Vec*>(src + e);
                Vec hi = *reinterpret_cast<const Vec*>(src + half + e);
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    const float2 r = a[e + j];
                    const float p = as_f32(lo.v[j]), s = as_f32(hi.v[j]);
                    lo.v[j] = from_f32<T>(p * r.x - s * r.y);
                    hi.v[j] = from_f32<T>(p * r.y + s * r.x);
                }
                *reinterpret_cast<Vec*>(dst + e) = lo;
                *reinterpret_cast<Vec*>(dst + half + e) = hi;
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
    bool vec = a.dh * sizeof(T) % 16 == 0 && a.rot * sizeof(T) % (a.interleaved ? 16 : 32) == 0;
    const void* ptr[4] = {a.q, a.k, a.qo, a.ko};
    for (int i = 0; i < 8; ++i) {
        g.s[i] = a.strides[i];
        if ((i / 2) % 2 && !a.Hkv) continue;
        vec = vec && a.strides[i] * (int64_t)sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(ptr[i / 2]) % 16 == 0;
    }
    g.copy_tail = a.rot < a.dh && (a.q != a.qo || (a.Hkv && a.k != a.ko));
    // As many tokens a round as leave every SM a few CTAs; a step of few tokens is split
    // over the heads, each CTA with its own sines.
    const int heads = a.H + a.Hkv, want = sm_count() * 4;
    g.tokens = kRopeTokens;
    while (g.tokens > 1 && (a.T + g.tokens - 1) / g.tokens < want) g.tokens >>= 1;
    const int chunks = (a.T + g.tokens - 1) / g.tokens;
    g.head_splits = chunks >= want / 2 ? 1 : (want / 2 + chunks - 1) / chunks;
    if (g.head_splits > heads) g.head_splits = heads;
    g.heads_per = (heads + g.head_splits - 1) / g.head_splits;
    g.head_splits = (heads + g.heads_per - 1) / g.heads_per;
    const int cap = sm_count() * 8, rounds = (chunks + cap - 1) / cap;
    const dim3 grid((chunks + rounds - 1) / rounds, g.head_splits);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(kRopeThreads), 0, st, static_cast<const T*>(a.q),
                          static_cast<const T*>(a.k), static_cast<T*>(a.qo), static_cast<T*>(a.ko), a.positions,
                          a.inv_freq, g);
    };
    if (vec) return a.interleaved ? go(k_rope_rows<T, true, true>) : go(k_rope_rows<T, true, false>);
    return a.interleaved ? go(k_rope_rows<T, false, true>) : go(k_rope_rows<T, false, false>);
}

}  // namespace

cudaError_t launch_rope_rows(const RopeRowsArgs& a, cudaStream_t st) {
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace tfm
