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
// 64 sequences of 5 drafted tokens and 50257 logits take 35 us: the first launch 23, bound by
// reading the logits (127 MB); decisions and race, bound by their chains of dependent
// loads and by the race's ~50 instructions per logit, the rest.  One sequence of 4 and 32000
// takes 9 us, the latency of two launches.
//
// Both decisions compare computed numbers, so a rounding may turn them.  Each is made
// in fp32 where the sides are further apart than their errors (kEps), else in fp64 with
// the rows' sums as the first launch left them, in fp32 per chunk (kEpsSum).  Where that
// leaves it open too, by the bounds' widths in one of some 200 batches of 64 x 5 drafts, the CTA
// takes the rows' sums anew from the logits, as pairs of fp32 numbers (kEpsPair), and if
// those do not tell, in fp64.  In the race a weight p - q is known to eps (p + q); every chunk keeps
// what may still be its winner, or itself as a whole if the chunks' sums do not tell.
// (Without a refused token the sum scales all weights alike and decides nothing.)  Ties go
// to the lowest token.
#include <climits>

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
// of a row's sum that adds the chunks' in fp64: 3.0e-6, 20 roundings within a chunk
// and one exponential, 4.4e-6
constexpr double kEpsSum = 5e-6;
constexpr double kEpsPair = 1e-11;      // of a sum of pairs (pair_share)

struct __align__(16) Cand {
    float lo, hi;      // bounds of weight / noise
    int idx;           // the token; kNone, or kOpen: more than one of the chunk may be it
    int pad;
};
constexpr int kNone = -1, kOpen = -2;
constexpr int kMostOpen = 64;           // threads with candidates that fp64 looks at within a chunk

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
    double inv_temp;   // 1 / temperature (a division in fp64 costs the race's CTAs 8 us of 64 x 5 drafts)
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
__device__ __forceinline__ double weight64(float z, float m, double inv_temp) {
    if (z == m) return 1.0;
    return exp(fmax(((double)z - (double)m) * inv_temp, -1e300));
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

// A larger value wins, the lower index among equal ones; a negative index never wins.
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

// The block's best, in all threads.
__device__ __forceinline__ void block_best(double& v, int& i, double* redv, int* redi) {
    warp_best(v, i);
    if ((threadIdx.x & 31) == 0) {
        redv[threadIdx.x >> 5] = v;
        redi[threadIdx.x >> 5] = i;
    }
    __syncthreads();
    v = redv[0];
    i = redi[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) take_better(v, i, redv[w], redi[w]);
    __syncthreads();
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
// Its sum in fp64 from the chunks' in fp32 (kEpsSum), by one warp, a chunk a lane (the fp64
// units take 32 cycles an instruction: only where a decision needs it; by one thread it took
// 10 us and more, which two of ten batches of 64 x 5 drafts waited for: 52 and 58 us instead of 39,
// 40 and 46 now).
__device__ __noinline__ double row_sum64(const float2* __restrict__ part, int C, float m, double inv_temp) {
    double s = 0.0;
    if (m > -INFINITY)
        for (int c = threadIdx.x & 31; c < C; c += 32) s += (double)part[c].y * weight64(part[c].x, m, inv_temp);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// This thread's share of a row's sum from its logits (m finite), as pairs of fp32 numbers; `tab`
// holds 2^(k / 256) so.  The difference and its product with log2(e) / temperature are
// taken with their rounding errors: y = yh + yl, to 5e-13 for |y| <= 24.  With yh = k / 256 + g the weight is
// 2^(k / 256) (1 + h + h^2 / 2 + ...), h = (g + yl) ln 2, |h| < 1.4e-3, each product that counts taken with
// its error: ~1e-12 in all.  Two rows of 50257 logits take a CTA 85 us so, in fp64 ~800.
__device__ __noinline__ double pair_share(const float* __restrict__ row, int V, float m, double inv_temp,
                                          const float2* tab) {
    constexpr double kLn2 = 0.69314718055994530942;
    constexpr float kLn2Hi = (float)kLn2, kLn2Lo = (float)(kLn2 - (double)kLn2Hi);
    const double c = 1.4426950408889634 * inv_temp;
    const float ch = (float)c, cl = (float)(c - (double)ch);
    double total = 0.0;
    for (int v0 = threadIdx.x; v0 < V; v0 += 64 * kThreads) {
        float sum = 0.f, low = 0.f;                    // 64 weights: `low` stays small beside `sum`
        auto add = [&](float x) {
            const float t = __fadd_rn(sum, x), w = __fsub_rn(t, sum);
            low = __fadd_rn(low, __fadd_rn(__fsub_rn(sum, __fsub_rn(t, w)), __fsub_rn(x, w)));
            sum = t;
        };
        auto weigh = [&](float z) {
            const float d = __fsub_rn(z, m);
            if (!(d * ch > -80.f)) return;             // all of these together: below 2^-56 of the sum
            const float w = __fsub_rn(d, z);           // d + de = z - m
            const float de = __fsub_rn(__fsub_rn(z, __fsub_rn(d, w)), __fadd_rn(m, w));
            const float yh = __fmul_rn(d, ch);
            const float yl = __fadd_rn(__fmaf_rn(d, ch, -yh), __fmaf_rn(d, cl, __fmul_rn(de, ch)));
            const float n = rintf(yh * 256.f), g = __fmaf_rn(n, -1.f / 256.f, yh);
            const int k = (int)n;
            const float2 t = tab[k & 255];
            const float scale = __int_as_float(((k >> 8) + 127) << 23);
            const float hh = __fmul_rn(g, kLn2Hi);
            const float hl = __fadd_rn(__fmaf_rn(g, kLn2Hi, -hh), __fmaf_rn(g, kLn2Lo, __fmul_rn(yl, kLn2Hi)));
            const float r = hh * (hl + hh * (0.5f + hh * (1.f / 6.f + hh * (1.f / 24.f))));
            const float x = __fmul_rn(t.x, hh), xl = __fmaf_rn(t.x, hh, -x);
            add(t.x * scale);
            add(x * scale);
            low = __fmaf_rn(__fadd_rn(t.y, __fmaf_rn(t.x, __fadd_rn(hl, r), xl)), scale, low);
        };
        for (int v = v0; v < V && v < v0 + 64 * kThreads; v += 8 * kThreads) {
            float z[8];                                // asked for together
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = v + i * kThreads < V ? no_nan(__ldg(row + v + i * kThreads)) : -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) weigh(z[i]);
        }
        total += (double)sum + (double)low;
    }
    return total;
}
// The same in fp64; for any m.
__device__ __noinline__ double share64(const float* __restrict__ row, int V, float m, double inv_temp) {
    double s = 0.0;
    if (m > -INFINITY) {
#pragma unroll 4
        for (int v = threadIdx.x; v < V; v += kThreads) s += weight64(no_nan(row[v]), m, inv_temp);
    }
    return s;
}
// A row's sum from its logits, in all threads of the block.
struct SumSpace {
    float2 tab[256];
    double warp[kThreads / 32];
};
__device__ __noinline__ double logit_sum(const float* row, int V, float m, double inv_temp, bool exact, SumSpace& sp) {
    if (!exact) {
        const double t = exp2((double)threadIdx.x / 256.0);
        sp.tab[threadIdx.x] = make_float2((float)t, (float)(t - (double)(float)t));
        __syncthreads();
    }
    double s = exact || !(fabsf(m) < INFINITY) ? share64(row, V, m, inv_temp) : pair_share(row, V, m, inv_temp, sp.tab);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sp.warp[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += sp.warp[w];
    __syncthreads();
    return s;
}
static_assert(kThreads == 256, "a thread per entry of the table");
// p(z) or q(z) in fp64; 0 in a row without any weight.
__device__ __noinline__ double prob64(float z, float m, double sum, double inv_temp) {
    return sum > 0.0 ? weight64(z, m, inv_temp) / sum : 0.0;
}

// Whether token x is accepted, u q(x) < p(x), from the logits of both rows; by the block.  (Here and
// in settle_race out of line: within the kernels they cost 4.6 us of 35 where nothing is open.)
__device__ __noinline__ bool settle_draft(const float* __restrict__ trow, const float* __restrict__ drow, int V, int x,
                                          float u, float mt, float md, double inv_temp, SumSpace& sp) {
    for (int exact = 0;; ++exact) {
        const double st = logit_sum(trow, V, mt, inv_temp, exact, sp), sd = logit_sum(drow, V, md, inv_temp, exact, sp);
        const double p = prob64(no_nan(trow[x]), mt, st, inv_temp);
        const double uq = (double)u * prob64(no_nan(drow[x]), md, sd, inv_temp);
        if (exact || !(fabs(uq - p) < 2.0 * kEpsPair * p)) return uq < p;
    }
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
// What the chunks' sums leave open the whole CTA settles, in order, as far as it is reached.
__device__ __forceinline__ Decision decide(const VerifyParams& p, int b) {
    __shared__ float2 row_t[kMaxK + 1], row_d[kMaxK];     // maximum, sum
    __shared__ int take[kMaxK];                           // 0: refused, 1: accepted, 2: open
    __shared__ SumSpace space;
    const VerifyArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nd = drafted(a, b, nullptr);
    const double inv_temp = p.inv_temp;
    for (int i = warp; i <= nd; i += kThreads / 32) {
        const bool drafted_here = i < nd;
        const int x = drafted_here ? a.draft[(int64_t)b * a.K + i] : 0;
        const float u = drafted_here ? a.u[(int64_t)b * a.K + i] : 0.f;
        const float2* part_t = p.part + ((int64_t)b * (a.K + 1) + i) * p.C;
        const float2* part_d = p.part + ((int64_t)a.B * (a.K + 1) + (int64_t)b * a.K + i) * p.C;
        bool ok = drafted_here && x >= 0 && x < a.V, open = false;
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
                const double p64 = prob64(zt, mt, row_sum64(part_t, p.C, mt, inv_temp), inv_temp);
                const double uq64 = (double)u * prob64(zd, md, row_sum64(part_d, p.C, md, inv_temp), inv_temp);
                ok = uq64 < p64;
                open = fabs(uq64 - p64) < 2.0 * kEpsSum * p64;
            }
        }
        if (drafted_here && lane == 0) take[i] = open ? 2 : ok;
    }
    __syncthreads();
    int n = 0;
    for (; n < nd; ++n) {
        int ok = take[n];
        if (ok == 2) {
            ok = settle_draft(a.target + ((int64_t)b * (a.K + 1) + n) * a.ld_target,
                              a.dlogits + ((int64_t)b * a.K + n) * a.ld_draft, a.V, a.draft[(int64_t)b * a.K + n],
                              a.u[(int64_t)b * a.K + n], row_t[n].x, row_d[n].x, p.inv_temp, space);
        }
        if (!ok) break;
    }
    Decision d{};
    if (threadIdx.x == 0) {
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

// weight / noise of token v in fp64, and what a relative error of the sums is multiplied
// with there: (p + q) / noise; yrow null: of p alone.
__device__ __forceinline__ double race_score(const float* __restrict__ zrow, const float* __restrict__ yrow,
                                             const float* __restrict__ erow, int v, float mt, float md, double st,
                                             double sd, double inv_temp, double& mag) {
    mag = 0.0;
    const float ev = erow[v];
    if (!(ev > 0.f)) return 0.0;
    double w = prob64(no_nan(zrow[v]), mt, st, inv_temp);
    if (yrow) {
        const double q = prob64(no_nan(yrow[v]), md, sd, inv_temp);
        mag = (w + q) / (double)ev;
        w -= q;
    }
    return w / (double)ev;
}
__device__ __forceinline__ Cand load_cand(const int4* cd, int k) {     // from L2: other CTAs wrote them
    const int4 w = __ldcg(cd + k);
    return Cand{__int_as_float(w.x), __int_as_float(w.y), w.z, 0};
}
// The new token after a refused one, where the chunks' sums leave it open: the winner of the race over
// max(p - q, 0) with the sums from the logits, among the tokens and chunks whose upper bound
// reaches `from`; then, if the residual there is no more than fp32 holds (or `from` is inf: nothing
// is there), among all; then, if it is zero everywhere, the winner of the race over p.  By the block.
__device__ __noinline__ int settle_race(const float* __restrict__ zrow, const float* __restrict__ yrow,
                                        const float* __restrict__ erow, const int4* cd, int RC, int V, float mt, float md,
                                        float from, double inv_temp, SumSpace& sp, double* redv, int* redi) {
    bool all = !(from < INFINITY);
    for (int exact = all;; ++exact) {
        const double st = logit_sum(zrow, V, mt, inv_temp, exact, sp), sd = logit_sum(yrow, V, md, inv_temp, exact, sp);
        bool every = true;                             // were looked at
        double low = 0.0, high = 0.0, next = 0.0;      // bounds: the best lower one; the two best upper ones
        int best = kNone;
        for (int k = 0; k < RC; ++k) {
            const Cand x = load_cand(cd, k);
            const bool chunk = all || x.idx == kOpen, in = all || (x.idx != kNone && x.hi >= from && x.hi > 0.f);
            every = every && chunk && in;
            if (!in) continue;
            const int end = chunk ? min((k + 1) * kRaceChunk, V) : x.idx + 1;
            for (int i = (chunk ? k * kRaceChunk : x.idx) + (int)threadIdx.x; i < end; i += kThreads) {
                double mag;
                const double s = race_score(zrow, yrow, erow, i, mt, md, st, sd, inv_temp, mag);
                const double err = exact ? 0.0 : kEpsPair * mag, h = s + err;
                if (!(h > 0.0)) continue;
                low = fmax(low, s - err);
                next = fmax(next, fmin(high, h));
                take_better(high, best, h, i);
            }
        }
        if (!exact) {
            int who = low > 0.0 ? (int)threadIdx.x : kNone;
            block_best(low, who, redv, redi);          // the best lower bound
            const int left = __syncthreads_count(best >= 0 && high >= low);
            const int more = __syncthreads_or(next > 0.0 && next >= low);
            if (left > 1 || more || (left == 1 && who < 0)) continue;
        }
        block_best(high, best, redv, redi);
        if (best >= 0 && (every || high * (double)erow[best] > 0x1p-125)) return best;
        if (every) break;
        all = true;
        exact = 0;
    }
    double v = 0.0, mag;
    int token = kNone;
    for (int x = threadIdx.x; x < V; x += kThreads) {
        const double s = race_score(zrow, nullptr, erow, x, mt, md, 1.0, 0.0, inv_temp, mag);
        if (s > 0.0) take_better(v, token, s, x);
    }
    block_best(v, token, redv, redi);
    return token;
}

// kDecide: each CTA decides for itself (see launch_verify_draft).
template <bool kDecide>
__global__ void __launch_bounds__(kThreads, 4) k_verify_race(const VerifyParams p) {
    __shared__ float red[kThreads / 32];
    __shared__ double redv[kThreads / 32];
    __shared__ int redi[kThreads / 32];
    __shared__ int last;
    __shared__ SumSpace space;
    __shared__ double sums[2];                         // of the rows of p and q, in fp64
    __shared__ float open_from;                        // the bound of what the chunks' sums leave open
    pdl_wait();
    pdl_trigger();
    const VerifyArgs& a = p.a;
    const int c = (int)(blockIdx.x % (unsigned)p.RC), b = (int)(blockIdx.x / (unsigned)p.RC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const double inv_temp = p.inv_temp;
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
    auto score64 = [&](int v, bool with_q, double st64, double sd64, double& mag) -> double {
        return race_score(zrow, with_q ? yrow : nullptr, erow, v, mt, md, st64, sd64, inv_temp, mag);
    };
    // bounds in fp32 of a score in fp64
    auto below = [](double x) { return (float)x - kEps * fabsf((float)x); };
    auto above = [](double x) { return (float)x + kEps * fabsf((float)x); };
    auto sum_t64 = [&]() { return row_sum64(p.part + ((int64_t)b * (a.K + 1) + n) * p.C, p.C, mt, inv_temp); };
    auto sum_d64 = [&]() {
        return refused ? row_sum64(p.part + ((int64_t)a.B * (a.K + 1) + (int64_t)b * a.K + n) * p.C, p.C, md, inv_temp) : 0.0;
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
    } else if (!refused) {
        double v = 0.0;
        int best = kNone;
        if (any) {                                     // (the same in all threads)
            if (warp == 0) {
                const double t = sum_t64();
                if (lane == 0) sums[0] = t;
            }
            __syncthreads();
        }
        for (; mine; mine &= mine - 1) {
            const int idx = index_of<kRaceVec>(c, __ffs(mine) - 1);
            double mag;
            const double s = score64(idx, false, sums[0], 0.0, mag);
            if (s > 0.0) take_better(v, best, s, idx);
        }
        block_best(v, best, redv, redi);
        if (threadIdx.x == 0) *out = Cand{below(v), above(v), best, 0};
    } else if (any == 0 || any > kMostOpen) {
        top = block_max(top, red);
        if (threadIdx.x == 0) *out = Cand{lo, top, any ? kOpen : kNone, 0};
    } else {
        if (warp == 0) {
            const double t = sum_t64();
            if (lane == 0) sums[0] = t;
        } else if (warp == 1) {
            const double q = sum_d64();
            if (lane == 0) sums[1] = q;
        }
        __syncthreads();
        float low = -INFINITY, high = -INFINITY, next = -INFINITY;    // next: the second highest upper bound
        int best = kNone;
        for (; mine; mine &= mine - 1) {
            const int idx = index_of<kRaceVec>(c, __ffs(mine) - 1);
            double mag;
            const double s = score64(idx, true, sums[0], sums[1], mag), err = kEpsSum * mag;
            low = fmaxf(low, below(s - err));
            const float h = above(s + err);
            if (h > high) best = idx;
            next = fmaxf(next, fminf(high, h));
            high = fmaxf(high, h);
        }
        low = block_max(low, red);
        const bool may = high > 0.f && high >= low;
        const int left = __syncthreads_count(may), more = __syncthreads_or(next > 0.f && next >= low);
        if (left == 1 && !more) {
            if (may) *out = Cand{low, high, best, 0};
        } else {
            high = block_max(high, red);
            if (threadIdx.x == 0) *out = Cand{low, high, left ? kOpen : kNone, 0};
        }
    }
    // The last CTA of the sequence merges the chunks.
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.done + b, 1) == p.RC - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    int4* const cd = reinterpret_cast<int4*>(p.cand + (int64_t)b * p.RC);
    auto cand = [&](int k) { return load_cand(cd, k); };
    if (warp == 0) {
        float lb = -INFINITY;
        int only, total;
        auto contenders = [&]() {                      // how many, and the one if it is one
            int cnt = 0;
            only = INT_MIN;
            for (int k = lane; k < p.RC; k += 32) {
                const Cand x = cand(k);
                if (x.idx != kNone && x.hi >= lb) {
                    ++cnt;
                    only = x.idx;
                }
            }
            total = __reduce_add_sync(0xffffffffu, cnt);
            only = __reduce_max_sync(0xffffffffu, only);
        };
        for (int k = lane; k < p.RC; k += 32) {
            const Cand x = cand(k);
            if (x.idx != kNone) lb = fmaxf(lb, x.lo);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lb = fmaxf(lb, __shfl_xor_sync(0xffffffffu, lb, o));
        contenders();
        int token = kNone;
        bool open = false;
        if (total == 1 && only >= 0 && (!refused || lb > 0.f)) {
            token = only;
        } else if (total > 0) {
            const double st64 = sum_t64(), sd64 = sum_d64();
            double v = 0.0;
            float low = lb;
            for (int k = lane; k < p.RC; k += 32) {
                const Cand x = cand(k);
                if (x.idx < 0 || !(x.hi >= lb)) continue;
                double mag;
                const double s = score64(x.idx, true, st64, sd64, mag), err = kEpsSum * mag;
                take_better(v, token, s, x.idx);
                low = fmaxf(low, below(s - err));
                __stcg(cd + k, make_int4(__float_as_int(below(s - err)), __float_as_int(above(s + err)), x.idx, 0));
            }
            warp_best(v, token);
            if (refused) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) low = fmaxf(low, __shfl_xor_sync(0xffffffffu, low, o));
                lb = low;
                contenders();
                open = !(total == 1 && only >= 0 && lb > 0.f);
                token = open ? kNone : only;
            }
        }
        if (lane == 0) {
            redi[0] = token;
            open_from = open ? lb : INFINITY;
        }
    }
    __syncthreads();
    int token = redi[0];
    const float from = open_from;
    __syncthreads();
    if (refused && token < 0 && st > 0.f)
        token = settle_race(zrow, yrow, erow, cd, p.RC, a.V, mt, md, from, inv_temp, space, redv, redi);
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
    p.inv_temp = greedy ? 0.0 : 1.0 / (double)a.temperature;
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
