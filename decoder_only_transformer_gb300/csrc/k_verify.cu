// k_verify.cu - verification of drafted tokens against the target model's
// distribution.
//
// With p_i, q_i the softmax of the target's and the drafter's logits over
// z / temperature, drafted token x_i is accepted iff u_i q_i(x_i) < p_i(x_i) and
// every earlier one was.  At the first refusal the new token is drawn from
// max(p - q, 0), after the last accepted one from p; both by an exponential
// race, argmax_v weight(v) / noise(v), which needs no normalised sum of the
// weights and no running sum over the vocabulary.
//
// Three launches.  The first takes every row that can matter once through the SMs
// and leaves, per chunk of 8192 logits, the maximum m and the sum of
// e^((z - m) / temperature) (greedy: the largest logit and its index).  The second
// merges them, a CTA per sequence, and decides which tokens are accepted.  The third
// runs the race over the one row of p (and q) that is then needed, a CTA per chunk;
// the last CTA of a sequence to finish merges the chunks' winners and writes the
// answer.  A race of few CTAs decides itself, without the second launch; of many, each
// would repeat 13 chains of dependent loads.
// 64 sequences of 5 drafted tokens and 50257 logits take 36 us: the first launch 23, bound by
// reading the logits (127 MB); decisions and race, bound by their chains of dependent
// loads and by the race's ~50 instructions per logit, the rest.  One sequence of 4 and 32000
// takes 9 us, the latency of two launches.
//
// Both decisions compare computed numbers, so a rounding may turn them.  The
// acceptance test is done in fp32 where its two sides are further apart than
// their errors, else in fp64 from the merged statistics.  The race is run
// in fp32 with bounds: a weight p - q is known to kEps (p + q), every chunk
// keeps what may still be its winner, and where more than one token may be, those
// few are evaluated in fp64.  Ties go to the lowest token.
#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

constexpr int kThreads = 256;
// float4 loads per thread and logits per CTA: of the statistics (8 loads: at 4 the
// instructions a warp needs besides were half of all, 28 us instead of 23 for 64 x 11 rows of
// 50257), and of the race, which holds three rows' values
constexpr int kVec = 8, kRaceVec = 4;
constexpr int kChunk = kThreads * kVec * 4, kRaceChunk = kThreads * kRaceVec * 4;
constexpr int kMaxK = 64;
constexpr int kFewCtas = 128;           // of the race: it decides itself then
// Relative error of an fp32 probability.  The exponent x = (z - m) log2(e) / temperature
// carries three roundings (the factor, taken in fp64 on the host, the difference, the
// product), 3 * 2^-24 |x|, and so its weight 0.7 times that: 1.57e-5 down to the smallest
// normal number (|x| = 126).  A row's sum has the same error in its weights' exponents, |x|
// being at most log2(V) <= 24 on their average: 3.0e-6; 20 roundings within a chunk and up to 70
// over the chunks of 2^24 logits, 5.4e-6; the exponentials (2^-22 each, two in the sum), the
// division and the product with 1 / noise 1.2e-6.  2.6e-5 in all.
constexpr float kEps = 3e-5f;

struct __align__(16) Cand {
    float lo, hi;      // bounds of weight / noise
    int idx;           // -1: none
    int pad;
};

// What the race of a sequence is run over: the place of the new token, whether a
// drafted one was refused there, and both rows' statistics.
struct __align__(16) Decision {
    int n, refused;
    float mt, st, md, sd;
    int pad[2];
};

struct VerifyParams {
    VerifyArgs a;
    int C, RC;         // chunks per row: of the statistics, of the race
    float c2;          // log2(e) / temperature
    float2* part;      // [B*(K+1) + B*K][C]
    Cand* cand;        // [B][RC]
    Decision* dec;     // [B]
    int* done;         // [B] CTAs of a sequence that have finished
    int* err;
};

__device__ __forceinline__ float no_nan(float z) { return fmaxf(z, -INFINITY); }   // NaN -> -inf

// e^((z - m) / temperature) as an fp32 power of two; z = m gives 1 (also for an
// infinite m), a NaN exponent 0.  (2^-200 is 0: ex2.approx.ftz has no subnormal
// results, and a weight below 1e-38 of the largest one never decides.)
__device__ __forceinline__ float weight(float z, float m, float c2) {
    const float x = z == m ? 0.f : (z - m) * c2;
    return fast_exp2(fmaxf(x, -200.f));
}
__device__ __forceinline__ double weight64(float z, float m, double temperature) {
    if (z == m) return 1.0;
    return exp(fmax(((double)z - (double)m) / temperature, -1e300));
}

__device__ __forceinline__ int drafted(const VerifyArgs& a, int b, int* err) {
    int n = a.n_draft ? __ldg(a.n_draft + b) : a.K;
    if (n < 0 || n > a.K) {
        if (threadIdx.x == 0) raise_error(err, TFM_EINVAL);
        n = n < 0 ? 0 : a.K;
    }
    return n;
}

// The 4 N logits of this thread: chunk c of kThreads * 4 N, [j][e] at
// (j*kThreads + tid)*4 + e of it; `fill` behind the row's end.  ld is a multiple of 4
// and at least V, so a vector that starts inside the row lies inside its storage.
template <int N>
__device__ __forceinline__ void load_chunk(const float* __restrict__ row, int c, int V, float fill,
                                           float (&z)[4 * N]) {
    const int i0 = c * (kThreads * 4 * N) + (int)threadIdx.x * 4;
    const float4* src = reinterpret_cast<const float4*>(row + i0);
    float4 w[N];
    const bool whole = (c + 1) * (kThreads * 4 * N) <= V;
    if (whole) {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = __ldg(src + j * kThreads);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            w[j] = i0 + j * kThreads * 4 < V ? __ldg(src + j * kThreads) : make_float4(fill, fill, fill, fill);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        z[4 * j] = w[j].x;
        z[4 * j + 1] = w[j].y;
        z[4 * j + 2] = w[j].z;
        z[4 * j + 3] = w[j].w;
    }
    if (!whole) {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 1; e < 4; ++e)
                if (i0 + j * kThreads * 4 + e >= V) z[4 * j + e] = fill;
    }
}
template <int N>
__device__ __forceinline__ int index_of(int c, int k) {
    return c * (kThreads * 4 * N) + ((k >> 2) * kThreads + (int)threadIdx.x) * 4 + (k & 3);
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) v = fmaxf(v, red[w]);
    return v;
}

// A larger value wins, the lower index among equal ones; index -1 never wins.
template <typename F>
__device__ __forceinline__ void take_better(F& v, int& i, F v2, int i2) {
    if (i2 >= 0 && (i < 0 || v2 > v || (v2 == v && i2 < i))) {
        v = v2;
        i = i2;
    }
}
template <typename F>
__device__ __forceinline__ void warp_best(F& v, int& i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const F v2 = __shfl_xor_sync(0xffffffffu, v, o);
        const int i2 = __shfl_xor_sync(0xffffffffu, i, o);
        take_better(v, i, v2, i2);
    }
}

template <bool kGreedy>
__global__ void __launch_bounds__(kThreads) k_verify_stats(const VerifyParams p) {
    __shared__ float red[kThreads / 32];
    __shared__ float red2[kThreads / 32];
    __shared__ int redi[kThreads / 32];
    pdl_wait();
    pdl_trigger();
    const VerifyArgs& a = p.a;
    const int c = (int)(blockIdx.x % (unsigned)p.C), row = (int)(blockIdx.x / (unsigned)p.C);
    const int nt = a.B * (a.K + 1);
    const bool is_draft = row >= nt;
    const int r = is_draft ? row - nt : row;
    const int per = is_draft ? a.K : a.K + 1;
    const int b = r / per, i = r - b * per;
    const int nd = drafted(a, b, p.err);
    if (!kGreedy && !is_draft && i == 0 && c == 0 && threadIdx.x == 0) p.done[b] = 0;
    if (is_draft ? i >= nd : i > nd) return;          // a row nobody asks for
    float z[4 * kVec];
    load_chunk<kVec>(is_draft ? a.dlogits + (int64_t)r * a.ld_draft : a.target + (int64_t)r * a.ld_target, c, a.V,
           -INFINITY, z);
    // (a maximum with a NaN is the other operand)
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < 4 * kVec; k += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmax3(mx[e], z[k + 2 * e], z[k + 2 * e + 1]);
    float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float2* out = p.part + (int64_t)row * p.C + c;
    if (kGreedy) {
        int best = -1;
#pragma unroll
        for (int k = 4 * kVec - 1; k >= 0; --k)
            if (z[k] == m && m > -INFINITY) best = index_of<kVec>(c, k);
        warp_best(m, best);
        if (lane == 0) {
            red[warp] = m;
            redi[warp] = best;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) take_better(m, best, red[w], redi[w]);
            *out = make_float2(m, __int_as_float(best));
        }
        return;
    }
    m = block_max(m, red);
    float s = 0.f;
    if (m > -INFINITY && m < INFINITY) {
        // packed pairs: (z - m) c2, then the power; NaN and -inf end at the bound
        const uint64_t negm = f2_pack(-m, -m), c2 = f2_pack(p.c2, p.c2);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int k = 0; k < 4 * kVec; k += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_add(f2_pack(z[k], z[k + 1]), negm), c2, 0ull), x0, x1);
            sum[(k >> 1) & 1] = f2_add(sum[(k >> 1) & 1], f2_pack(fast_exp2(fmaxf(x0, -200.f)), fast_exp2(fmaxf(x1, -200.f))));
        }
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        s = s0 + s1;
    } else if (m == INFINITY) {                        // all the weight on the infinite ones
#pragma unroll
        for (int k = 0; k < 4 * kVec; ++k) s += z[k] == INFINITY ? 1.f : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red2[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = red2[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) s += red2[w];
        *out = make_float2(m, s);
    }
}

// The maximum and the sum of a whole row from its chunks, by one warp.  The maximum first:
// a sum that is scaled anew whenever the maximum grows takes an exponential's error each time.
__device__ __forceinline__ void row_stats(const float2* __restrict__ part, int C, float c2, float& m,
                                          float& s) {
    const int lane = threadIdx.x & 31;
    const float2 first = lane < C ? part[lane] : make_float2(-INFINITY, 0.f);
    m = first.x;
    s = 0.f;
    for (int c = lane + 32; c < C; c += 32) m = fmaxf(m, part[c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) return;
    s = first.y * weight(first.x, m, c2);
    for (int c = lane + 32; c < C; c += 32) {
        const float2 v = part[c];
        s += v.y * weight(v.x, m, c2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
}
// Its sum in fp64, by one warp, a chunk a lane (the fp64 units take 32 cycles an
// instruction: only where a decision needs it; by one thread it took 10 us and more, which
// two of ten batches of 64 x 5 drafts waited for: 52 and 58 us instead of 39, 40 and 46 now).
__device__ __noinline__ double row_sum64(const float2* __restrict__ part, int C, float m, double temperature) {
    double s = 0.0;
    if (m > -INFINITY)
        for (int c = threadIdx.x & 31; c < C; c += 32) s += (double)part[c].y * weight64(part[c].x, m, temperature);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// p(z) or q(z) in fp64; 0 in a row without any weight.
__device__ __noinline__ double prob64(float z, float m, double sum, double temperature) {
    return sum > 0.0 ? weight64(z, m, temperature) / sum : 0.0;
}

// tokens[b] and n_accepted[b]; called by one warp.
__device__ __forceinline__ void write_answer(const VerifyArgs& a, int b, int n, int token) {
    const int lane = threadIdx.x & 31;
    for (int i = lane; i <= a.K; i += 32)
        a.tokens[(int64_t)b * (a.K + 1) + i] = i < n ? a.draft[(int64_t)b * a.K + i] : i == n ? token : -1;
    if (lane == 0) a.n_accepted[b] = n;
}

// Which drafted tokens of sequence b are accepted: by a CTA, a warp per place; what
// does not depend on one another is asked for together.  The answer is thread 0's.
__device__ __forceinline__ Decision decide(const VerifyParams& p, int b) {
    __shared__ float2 row_t[kMaxK + 1], row_d[kMaxK];     // maximum, sum
    __shared__ int take[kMaxK];
    const VerifyArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nd = drafted(a, b, nullptr);
    const double temp = (double)a.temperature;
    for (int i = warp; i <= nd; i += kThreads / 32) {
        const bool drafted_here = i < nd;
        const int x = drafted_here ? a.draft[(int64_t)b * a.K + i] : 0;
        const float u = drafted_here ? a.u[(int64_t)b * a.K + i] : 0.f;
        const float2* part_t = p.part + ((int64_t)b * (a.K + 1) + i) * p.C;
        const float2* part_d = p.part + ((int64_t)a.B * (a.K + 1) + (int64_t)b * a.K + i) * p.C;
        bool ok = drafted_here && x >= 0 && x < a.V;
        if (drafted_here && !ok && lane == 0) raise_error(p.err, TFM_EBADTOKEN);
        float zt = 0.f, zd = 0.f;
        if (ok) {
            zt = no_nan(a.target[((int64_t)b * (a.K + 1) + i) * a.ld_target + x]);
            zd = no_nan(a.dlogits[((int64_t)b * a.K + i) * a.ld_draft + x]);
        }
        float mt, md = 0.f, st, sd = 0.f;
        row_stats(part_t, p.C, p.c2, mt, st);
        if (drafted_here) row_stats(part_d, p.C, p.c2, md, sd);
        // (the lanes' sums may differ in the last bit; one decides for all)
        st = __shfl_sync(0xffffffffu, st, 0);
        sd = __shfl_sync(0xffffffffu, sd, 0);
        if (lane == 0) {
            row_t[i] = make_float2(mt, st);
            if (drafted_here) row_d[i] = make_float2(md, sd);
        }
        if (ok) {
            const float px = st > 0.f ? weight(zt, mt, p.c2) / st : 0.f;
            const float uq = u * (sd > 0.f ? weight(zd, md, p.c2) / sd : 0.f);
            // fp32 decides where the two sides are further apart than their errors (and not
            // lost below its normal numbers); the same in all lanes
            if (px > 1e-30f && uq * (1.f + 2.f * kEps) < px * (1.f - 2.f * kEps)) {
                ok = true;
            } else if (uq > 1e-30f && uq * (1.f - 2.f * kEps) > px * (1.f + 2.f * kEps)) {
                ok = false;
            } else {
                const double p64 = prob64(zt, mt, row_sum64(part_t, p.C, mt, temp), temp);
                const double q64 = prob64(zd, md, row_sum64(part_d, p.C, md, temp), temp);
                ok = (double)u * q64 < p64;
            }
        }
        if (drafted_here && lane == 0) take[i] = ok;
    }
    __syncthreads();
    Decision d{};
    if (threadIdx.x == 0) {
        int n = 0;
        while (n < nd && take[n]) ++n;
        const bool refused = n < nd;
        d = Decision{n, refused, row_t[n].x, row_t[n].y, refused ? row_d[n].x : 0.f, refused ? row_d[n].y : 0.f, {0, 0}};
    }
    return d;
}
__global__ void __launch_bounds__(kThreads) k_verify_decide(const VerifyParams p) {
    pdl_wait();
    pdl_trigger();
    const Decision d = decide(p, (int)blockIdx.x);
    if (threadIdx.x == 0) p.dec[blockIdx.x] = d;
}

// kDecide: each CTA decides for itself (see launch_verify_draft).
template <bool kDecide>
__global__ void __launch_bounds__(kThreads, 4) k_verify_race(const VerifyParams p) {
    __shared__ float red[kThreads / 32];
    __shared__ double redv[kThreads / 32];
    __shared__ int redi[kThreads / 32];
    __shared__ int last;
    __shared__ double sums[2];                         // of the rows of p and q, in fp64
    pdl_wait();
    pdl_trigger();
    const VerifyArgs& a = p.a;
    const int c = (int)(blockIdx.x % (unsigned)p.RC), b = (int)(blockIdx.x / (unsigned)p.RC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const double temp = (double)a.temperature;
    const float* erow = a.noise + (int64_t)b * a.ld_noise;
    float e[4 * kRaceVec];
    load_chunk<kRaceVec>(erow, c, a.V, 0.f, e);        // needed whatever the row is
    __shared__ Decision own;
    if (kDecide) {
        const Decision mine = decide(p, b);
        if (threadIdx.x == 0) own = mine;
        __syncthreads();
    }
    const Decision d = kDecide ? own : p.dec[b];
    const int n = d.n;
    const bool refused = d.refused;
    const float mt = d.mt, st = d.st, md = d.md, sd = d.sd;
    const float inv_t = st > 0.f ? 1.f / st : 0.f, inv_d = sd > 0.f ? 1.f / sd : 0.f;
    const float* zrow = a.target + ((int64_t)b * (a.K + 1) + n) * a.ld_target;
    const float* yrow = refused ? a.dlogits + ((int64_t)b * a.K + n) * a.ld_draft : nullptr;
    // weight / noise of token v in fp64; with_q false: of p alone
    auto score64 = [&](int v, bool with_q, double st64, double sd64) -> double {
        const float ev = erow[v];
        if (!(ev > 0.f)) return 0.0;
        double w = prob64(no_nan(zrow[v]), mt, st64, temp);
        if (with_q && yrow) w -= prob64(no_nan(yrow[v]), md, sd64, temp);
        return w / (double)ev;
    };
    auto sum_t64 = [&]() { return row_sum64(p.part + ((int64_t)b * (a.K + 1) + n) * p.C, p.C, mt, temp); };
    auto sum_d64 = [&]() {
        return refused ? row_sum64(p.part + ((int64_t)a.B * (a.K + 1) + (int64_t)b * a.K + n) * p.C, p.C, md, temp) : 0.0;
    };
    float hi[4 * kRaceVec];
    float lo = -INFINITY;
    {
        float z[4 * kRaceVec], y[4 * kRaceVec];
        load_chunk<kRaceVec>(zrow, c, a.V, -INFINITY, z);
        if (refused) load_chunk<kRaceVec>(yrow, c, a.V, -INFINITY, y);
        if (fabsf(mt) < INFINITY && (!refused || fabsf(md) < INFINITY)) {
            // finite maxima: packed pairs, the exponents as in k_verify_stats (one at a time
            // and for any maximum 64 x 50257 took 38.7 us in all, this way 36.4)
            const uint64_t c2 = f2_pack(p.c2, p.c2), nmt = f2_pack(-mt, -mt), nmd = f2_pack(-md, -md);
            const uint64_t it = f2_pack(inv_t, inv_t), nid = f2_pack(-inv_d, -inv_d), minus = f2_pack(-1.f, -1.f);
            const uint64_t eps = f2_pack(kEps, kEps), neps = f2_pack(-kEps, -kEps);
            auto weights = [&](float a, float b, uint64_t neg_m, uint64_t scale) {
                float x0, x1;
                f2_unpack(f2_fma(f2_add(f2_pack(a, b), neg_m), c2, 0ull), x0, x1);
                return f2_fma(f2_pack(fast_exp2(fmaxf(x0, -200.f)), fast_exp2(fmaxf(x1, -200.f))), scale, 0ull);
            };
#pragma unroll
            for (int k = 0; k < 4 * kRaceVec; k += 2) {
                const uint64_t pw = weights(z[k], z[k + 1], nmt, it);
                const uint64_t nq = refused ? weights(y[k], y[k + 1], nmd, nid) : 0ull;       // -q
                const uint64_t r = f2_add(pw, nq), sum = f2_fma(nq, minus, pw);
                const uint64_t inv_e = f2_pack(__fdividef(1.f, e[k]), __fdividef(1.f, e[k + 1]));
                float p0, p1, h0, h1, l0, l1;
                f2_unpack(pw, p0, p1);
                f2_unpack(f2_fma(f2_fma(sum, eps, r), inv_e, 0ull), h0, h1);
                f2_unpack(f2_fma(f2_fma(sum, neps, r), inv_e, 0ull), l0, l1);
                const bool in0 = p0 > 0.f && e[k] > 0.f, in1 = p1 > 0.f && e[k + 1] > 0.f;
                hi[k] = in0 ? h0 : -INFINITY;
                hi[k + 1] = in1 ? h1 : -INFINITY;
                lo = fmax3(lo, in0 ? l0 : -INFINITY, in1 ? l1 : -INFINITY);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4 * kRaceVec; ++k) {
                const float pw = st > 0.f ? weight(no_nan(z[k]), mt, p.c2) * inv_t : 0.f;
                const float qw = refused && sd > 0.f ? weight(no_nan(y[k]), md, p.c2) * inv_d : 0.f;
                const bool in = pw > 0.f && e[k] > 0.f;
                const float r = pw - qw, er = kEps * (pw + qw), inv_e = __fdividef(1.f, e[k]);
                hi[k] = in ? (r + er) * inv_e : -INFINITY;
                lo = fmaxf(lo, in ? (r - er) * inv_e : -INFINITY);
            }
        }
    }
    lo = block_max(lo, red);
    uint32_t mine = 0;                                 // this thread's possible winners, as bits
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 4 * kRaceVec; ++k)
        if (hi[k] > 0.f && hi[k] >= lo) {
            mine |= 1u << k;
            top = fmaxf(top, hi[k]);
        }
    // how many may be the chunk's winner: 0, 1, or more
    const int any = __syncthreads_count(mine != 0), several = __syncthreads_or(mine & (mine - 1));
    Cand* out = p.cand + (int64_t)b * p.RC + c;
    if (any == 1 && !several && lo > 0.f) {
        if (mine) *out = Cand{lo, top, index_of<kRaceVec>(c, __ffs(mine) - 1), 0};
    } else {
        double v = 0.0;
        int best = -1;
        if (any) {                                     // (the same in all threads)
            if (warp == 0) {
                const double t = sum_t64();
                if (lane == 0) sums[0] = t;
            } else if (warp == 1) {
                const double q = sum_d64();
                if (lane == 0) sums[1] = q;
            }
            __syncthreads();
        }
        if (mine) {
            const double st64 = sums[0], sd64 = sums[1];
            for (; mine; mine &= mine - 1) {
                const int idx = index_of<kRaceVec>(c, __ffs(mine) - 1);
                const double s = score64(idx, true, st64, sd64);
                if (s > 0.0) take_better(v, best, s, idx);
            }
        }
        warp_best(v, best);
        if (lane == 0) {
            redv[warp] = v;
            redi[warp] = best;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) take_better(v, best, redv[w], redi[w]);
            // the winner's bounds: fp64 to fp32 and back
            *out = Cand{(float)v * (1.f - kEps), (float)v * (1.f + kEps), best, 0};
        }
    }
    // The last CTA of the sequence merges the chunks.
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.done + b, 1) == p.RC - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    double v = 0.0;
    int token = -1;
    if (warp == 0) {
        const int4* cd = reinterpret_cast<const int4*>(p.cand + (int64_t)b * p.RC);
        auto cand = [&](int k) {                       // from L2: other CTAs wrote them
            const int4 w = __ldcg(cd + k);
            return Cand{__int_as_float(w.x), __int_as_float(w.y), w.z, 0};
        };
        float lb = -INFINITY;
        for (int k = lane; k < p.RC; k += 32) {
            const Cand x = cand(k);
            if (x.idx >= 0) lb = fmaxf(lb, x.lo);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lb = fmaxf(lb, __shfl_xor_sync(0xffffffffu, lb, o));
        int cnt = 0, only = -1;
        for (int k = lane; k < p.RC; k += 32) {
            const Cand x = cand(k);
            if (x.idx >= 0 && x.hi >= lb) {
                ++cnt;
                only = x.idx;
            }
        }
        const int total = __reduce_add_sync(0xffffffffu, cnt);
        if (total == 1) {
            token = __reduce_max_sync(0xffffffffu, only);
        } else if (total > 1) {
            const double st64 = sum_t64(), sd64 = sum_d64();
            for (int k = lane; k < p.RC; k += 32) {
                const Cand x = cand(k);
                if (x.idx >= 0 && x.hi >= lb) take_better(v, token, score64(x.idx, true, st64, sd64), x.idx);
            }
            warp_best(v, token);
        }
        if (lane == 0) redi[0] = token;
    }
    __syncthreads();
    token = redi[0];
    __syncthreads();
    if (token < 0 && refused) {
        // max(p - q, 0) is zero everywhere: the race over p, in fp64
        v = 0.0;
        const double st64 = sum_t64();
        for (int x = threadIdx.x; x < a.V; x += kThreads) {
            const double s = score64(x, false, st64, 0.0);
            if (s > 0.0) take_better(v, token, s, x);
        }
        warp_best(v, token);
        if (lane == 0) {
            redv[warp] = v;
            redi[warp] = token;
        }
        __syncthreads();
        if (warp == 0)
            for (int w = 0; w < kThreads / 32; ++w) take_better(v, token, redv[w], redi[w]);
    }
    if (warp == 0) write_answer(a, b, n, token);
}

// Greedy: one warp per sequence.
__global__ void __launch_bounds__(kThreads) k_verify_greedy(const VerifyParams p) {
    pdl_wait();
    pdl_trigger();
    const VerifyArgs& a = p.a;
    const int b = (int)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= a.B) return;
    const int nd = drafted(a, b, nullptr);
    int n = 0, best;
    while (true) {
        const float2* part = p.part + ((int64_t)b * (a.K + 1) + n) * p.C;
        float m = -INFINITY;
        best = -1;
        for (int c = lane; c < p.C; c += 32) take_better(m, best, part[c].x, __float_as_int(part[c].y));
        warp_best(m, best);
        if (n == nd) break;
        const int x = a.draft[(int64_t)b * a.K + n];
        if ((x < 0 || x >= a.V) && lane == 0) raise_error(p.err, TFM_EBADTOKEN);
        if (x != best || best < 0) break;
        ++n;
    }
    write_answer(a, b, n, best);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t verify_workspace_bytes(int B, int K, int V) {
    const size_t C = ((size_t)V + kChunk - 1) / kChunk, RC = ((size_t)V + kRaceChunk - 1) / kRaceChunk;
    return align256((size_t)B * (2 * K + 1) * C * sizeof(float2)) + align256((size_t)B * RC * sizeof(Cand)) +
           align256((size_t)B * sizeof(Decision)) + align256((size_t)B * 4);
}

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t st) {
    VerifyParams p{};
    p.a = a;
    p.C = (a.V + kChunk - 1) / kChunk;
    p.RC = (a.V + kRaceChunk - 1) / kRaceChunk;
    const bool greedy = a.temperature == 0.f;
    p.c2 = greedy ? 0.f : (float)(1.4426950408889634 / (double)a.temperature);
    uint8_t* w = static_cast<uint8_t*>(a.ws);
    p.part = reinterpret_cast<float2*>(w);
    w += align256((size_t)a.B * (2 * a.K + 1) * p.C * sizeof(float2));
    p.cand = reinterpret_cast<Cand*>(w);
    w += align256((size_t)a.B * p.RC * sizeof(Cand));
    p.dec = reinterpret_cast<Decision*>(w);
    w += align256((size_t)a.B * sizeof(Decision));
    p.done = reinterpret_cast<int*>(w);
    p.err = device_error_word();
    const unsigned rows = (unsigned)(a.B * (greedy ? a.K + 1 : 2 * a.K + 1));
    cudaError_t e = greedy ? launch_pdl(k_verify_stats<true>, dim3(rows * p.C), dim3(kThreads), 0, st, p)
                           : launch_pdl(k_verify_stats<false>, dim3(rows * p.C), dim3(kThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    if (greedy) return launch_pdl(k_verify_greedy, dim3((a.B + 7) / 8), dim3(kThreads), 0, st, p);
    // Few CTAs: they decide themselves, all at once, which saves a launch (one sequence of
    // 4 drafted tokens and 32000 logits: 0.8 us of 10).  Many: a CTA per sequence
    // decides first (16 of 4 and 50257: 15.9 us instead of 17.4, 64 of 5: 46 instead of 51).
    const dim3 race((unsigned)(a.B * p.RC));
    if ((int64_t)a.B * p.RC <= kFewCtas) return launch_pdl(k_verify_race<true>, race, dim3(kThreads), 0, st, p);
    e = launch_pdl(k_verify_decide, dim3((unsigned)a.B), dim3(kThreads), 0, st, p);
    return e != cudaSuccess ? e : launch_pdl(k_verify_race<false>, race, dim3(kThreads), 0, st, p);
}

}  // namespace tfm
