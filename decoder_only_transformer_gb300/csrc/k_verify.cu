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
// Two launches.  The first takes every row that can matter once through the SMs
// and leaves, per chunk of 4096 logits, the maximum m and the sum of
// e^((z - m) / temperature) (greedy: the largest logit and its index).  The
// second merges them per sequence, decides which tokens are accepted, and runs
// the race over the one row of p (and q) that it then needs, a CTA per chunk;
// the last CTA of a sequence to finish merges the chunks' winners and writes the
// answer.  Bound by reading the logits.
//
// Both decisions compare computed numbers, so a rounding may turn them.  The
// acceptance test is done in fp64 from the merged statistics.  The race is run
// in fp32 with bounds: a weight p - q is known to kEps (p + q), every chunk
// keeps what may still be its winner, and where more than one token may be, those
// few are evaluated in fp64.  Ties go to the lowest token.
#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;                                   // float4 loads per thread
constexpr int kChunk = kThreads * kVec * 4;               // logits per CTA
constexpr int kMaxK = 64;
// Relative error of an fp32 weight e^((z - m) / temperature): the exponent
// x = (z - m) log2(e) / temperature carries three roundings, 3 * 2^-24 |x|, so
// the weight 0.7 * 3 * 2^-24 |x| <= 1.6e-5 down to the smallest normal number
// (|x| = 126); the sums and the exponential itself stay below 1e-6.
constexpr float kEps = 2e-5f;

struct __align__(16) Cand {
    float lo, hi;      // bounds of weight / noise
    int idx;           // -1: none
    int pad;
};

struct VerifyParams {
    VerifyArgs a;
    int C;             // chunks per row
    float c2;          // log2(e) / temperature
    float2* part;      // [B*(K+1) + B*K][C]
    Cand* cand;        // [B][C]
    int* done;         // [B] CTAs of a sequence that have finished
    int* err;
};

__device__ __forceinline__ float no_nan(float z) { return fmaxf(z, -INFINITY); }   // NaN -> -inf

// e^((z - m) / temperature) as an fp32 power of two; z = m gives 1 (also for an
// infinite m), a NaN exponent 0.
__device__ __forceinline__ float weight(float z, float m, float c2) {
    const float x = z == m ? 0.f : (z - m) * c2;
    return exp2f(fmaxf(x, -INFINITY));
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

// 16 logits of this thread: chunk c, [j][e] at c*kChunk + (j*kThreads + tid)*4 + e;
// `fill` behind the row's end.  ld is a multiple of 4 and at least V, so a vector
// that starts inside the row lies inside its storage.
__device__ __forceinline__ void load16(const float* __restrict__ row, int c, int V, float fill,
                                       float (&z)[16]) {
    float4 w[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int64_t i = (int64_t)c * kChunk + (j * kThreads + (int)threadIdx.x) * 4;
        w[j] = i < V ? __ldg(reinterpret_cast<const float4*>(row + i)) : make_float4(fill, fill, fill, fill);
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int64_t i = (int64_t)c * kChunk + (j * kThreads + (int)threadIdx.x) * 4;
        z[4 * j] = w[j].x;
        z[4 * j + 1] = i + 1 < V ? w[j].y : fill;
        z[4 * j + 2] = i + 2 < V ? w[j].z : fill;
        z[4 * j + 3] = i + 3 < V ? w[j].w : fill;
    }
}
__device__ __forceinline__ int index16(int c, int k) {
    return c * kChunk + ((k >> 2) * kThreads + (int)threadIdx.x) * 4 + (k & 3);
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
    if (!is_draft && i == 0 && c == 0 && threadIdx.x == 0) p.done[b] = 0;
    const int nd = drafted(a, b, p.err);
    if (is_draft ? i >= nd : i > nd) return;          // a row nobody asks for
    float z[16];
    load16(is_draft ? a.dlogits + (int64_t)r * a.ld_draft : a.target + (int64_t)r * a.ld_target, c, a.V,
           -INFINITY, z);
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        z[k] = no_nan(z[k]);
        m = fmaxf(m, z[k]);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float2* out = p.part + (int64_t)row * p.C + c;
    if (kGreedy) {
        int best = -1;
#pragma unroll
        for (int k = 15; k >= 0; --k)
            if (z[k] == m && m > -INFINITY) best = index16(c, k);
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
    if (m > -INFINITY) {
#pragma unroll
        for (int k = 0; k < 16; ++k) s += weight(z[k], m, p.c2);
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

// The maximum and the sum of a whole row from its chunks, by one warp.
__device__ __forceinline__ void row_stats(const float2* __restrict__ part, int C, float c2, float& m,
                                          double& s) {
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
    for (int c = lane; c < C; c += 32) m = fmaxf(m, part[c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    s = 0.0;
    if (m > -INFINITY)
        for (int c = lane; c < C; c += 32) s += (double)part[c].y * (double)weight(part[c].x, m, c2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
}

// tokens[b] and n_accepted[b]; called by one thread.
__device__ __forceinline__ void write_answer(const VerifyArgs& a, int b, int n, int token) {
    for (int i = 0; i <= a.K; ++i)
        a.tokens[(int64_t)b * (a.K + 1) + i] = i < n ? a.draft[(int64_t)b * a.K + i] : i == n ? token : -1;
    a.n_accepted[b] = n;
}

__global__ void __launch_bounds__(kThreads) k_verify_race(const VerifyParams p) {
    __shared__ float m_t[kMaxK + 1], m_d[kMaxK];
    __shared__ double s_t[kMaxK + 1], s_d[kMaxK];
    __shared__ int take[kMaxK];
    __shared__ float red[kThreads / 32];
    __shared__ double redv[kThreads / 32];
    __shared__ int redi[kThreads / 32];
    __shared__ int last;
    pdl_wait();
    pdl_trigger();
    const VerifyArgs& a = p.a;
    const int c = (int)(blockIdx.x % (unsigned)p.C), b = (int)(blockIdx.x / (unsigned)p.C);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nd = drafted(a, b, nullptr);
    const double temp = (double)a.temperature;
    // Statistics and acceptance of every place, a warp each.
    for (int i = warp; i <= nd; i += kThreads / 32) {
        float mt, md = 0.f;
        double st, sd = 0.0;
        row_stats(p.part + ((int64_t)b * (a.K + 1) + i) * p.C, p.C, p.c2, mt, st);
        if (i < nd) row_stats(p.part + ((int64_t)a.B * (a.K + 1) + (int64_t)b * a.K + i) * p.C, p.C, p.c2, md, sd);
        if (lane == 0) {
            m_t[i] = mt;
            s_t[i] = st;
            if (i < nd) {
                m_d[i] = md;
                s_d[i] = sd;
                const int x = a.draft[(int64_t)b * a.K + i];
                bool ok = x >= 0 && x < a.V;
                if (!ok && c == 0) raise_error(p.err, TFM_EBADTOKEN);
                if (ok) {
                    const float zt = no_nan(a.target[((int64_t)b * (a.K + 1) + i) * a.ld_target + x]);
                    const float zd = no_nan(a.dlogits[((int64_t)b * a.K + i) * a.ld_draft + x]);
                    const double px = st > 0.0 ? weight64(zt, mt, temp) / st : 0.0;
                    const double qx = sd > 0.0 ? weight64(zd, md, temp) / sd : 0.0;
                    ok = (double)a.u[(int64_t)b * a.K + i] * qx < px;
                }
                take[i] = ok;
            }
        }
    }
    __syncthreads();
    int n = 0;
    while (n < nd && take[n]) ++n;
    const bool refused = n < nd;
    const float mt = m_t[n], md = refused ? m_d[n] : 0.f;
    const double st = s_t[n], sd = refused ? s_d[n] : 0.0;
    const float inv_t = st > 0.0 ? (float)(1.0 / st) : 0.f, inv_d = sd > 0.0 ? (float)(1.0 / sd) : 0.f;
    const float* zrow = a.target + ((int64_t)b * (a.K + 1) + n) * a.ld_target;
    const float* yrow = refused ? a.dlogits + ((int64_t)b * a.K + n) * a.ld_draft : nullptr;
    const float* erow = a.noise + (int64_t)b * a.ld_noise;
    // weight / noise of token v in fp64; with_q false: of p alone
    auto score64 = [&](int v, bool with_q) -> double {
        const float e = erow[v];
        if (!(e > 0.f) || !(st > 0.0)) return 0.0;
        double w = weight64(no_nan(zrow[v]), mt, temp) / st;
        if (with_q && yrow && sd > 0.0) w -= weight64(no_nan(yrow[v]), md, temp) / sd;
        return w / (double)e;
    };
    float hi[16];
    float lo = -INFINITY;
    {
        float z[16], y[16], e[16];
        load16(zrow, c, a.V, -INFINITY, z);
        load16(erow, c, a.V, 0.f, e);
        if (refused) load16(yrow, c, a.V, -INFINITY, y);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float pw = st > 0.0 ? weight(no_nan(z[k]), mt, p.c2) * inv_t : 0.f;
            const float qw = refused && sd > 0.0 ? weight(no_nan(y[k]), md, p.c2) * inv_d : 0.f;
            const bool in = pw > 0.f && e[k] > 0.f;
            const float r = pw - qw, er = kEps * (pw + qw);
            hi[k] = in ? (r + er) / e[k] : -INFINITY;
            lo = fmaxf(lo, in ? (r - er) / e[k] : -INFINITY);
        }
    }
    lo = block_max(lo, red);
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) mine += hi[k] > 0.f && hi[k] >= lo;
    // how many may be the chunk's winner: 0, 1, or more
    const int any = __syncthreads_count(mine > 0), several = __syncthreads_or(mine > 1);
    Cand* out = p.cand + (int64_t)b * p.C + c;
    if (any == 1 && !several && lo > 0.f) {
        if (mine) {
            int best = -1;
            float h = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (hi[k] > 0.f && hi[k] >= lo) {
                    best = index16(c, k);
                    h = hi[k];
                }
            *out = Cand{lo, h, best, 0};
        }
    } else {
        double v = 0.0;
        int best = -1;
        if (mine) {
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
                float h = hi[0];
#pragma unroll
                for (int kk = 1; kk < 16; ++kk)
                    if (kk == k) h = hi[kk];
                if (!(h > 0.f && h >= lo)) continue;
                const int idx = index16(c, k);
                const double s = score64(idx, true);
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
    if (threadIdx.x == 0) last = atomicAdd(p.done + b, 1) == p.C - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    double v = 0.0;
    int token = -1;
    if (warp == 0) {
        const int4* cd = reinterpret_cast<const int4*>(p.cand + (int64_t)b * p.C);
        auto cand = [&](int k) {                       // from L2: other CTAs wrote them
            const int4 w = __ldcg(cd + k);
            return Cand{__int_as_float(w.x), __int_as_float(w.y), w.z, 0};
        };
        float lb = -INFINITY;
        for (int k = lane; k < p.C; k += 32) {
            const Cand x = cand(k);
            if (x.idx >= 0) lb = fmaxf(lb, x.lo);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lb = fmaxf(lb, __shfl_xor_sync(0xffffffffu, lb, o));
        int cnt = 0, only = -1;
        for (int k = lane; k < p.C; k += 32) {
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
            for (int k = lane; k < p.C; k += 32) {
                const Cand x = cand(k);
                if (x.idx >= 0 && x.hi >= lb) take_better(v, token, score64(x.idx, true), x.idx);
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
        for (int x = threadIdx.x; x < a.V; x += kThreads) {
            const double s = score64(x, false);
            if (s > 0.0) take_better(v, token, s, x);
        }
        warp_best(v, token);
        if (lane == 0) {
            redv[warp] = v;
            redi[warp] = token;
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int w = 1; w < kThreads / 32; ++w) take_better(v, token, redv[w], redi[w]);
    }
    if (threadIdx.x == 0) write_answer(a, b, n, token);
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
    if (lane == 0) write_answer(a, b, n, best);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t verify_workspace_bytes(int B, int K, int V) {
    const size_t C = ((size_t)V + kChunk - 1) / kChunk;
    return align256((size_t)B * (2 * K + 1) * C * sizeof(float2)) + align256((size_t)B * C * sizeof(Cand)) +
           align256((size_t)B * 4);
}

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t st) {
    VerifyParams p{};
    p.a = a;
    p.C = (a.V + kChunk - 1) / kChunk;
    const bool greedy = a.temperature == 0.f;
    p.c2 = greedy ? 0.f : 1.4426950408889634f / a.temperature;
    uint8_t* w = static_cast<uint8_t*>(a.ws);
    p.part = reinterpret_cast<float2*>(w);
    w += align256((size_t)a.B * (2 * a.K + 1) * p.C * sizeof(float2));
    p.cand = reinterpret_cast<Cand*>(w);
    w += align256((size_t)a.B * p.C * sizeof(Cand));
    p.done = reinterpret_cast<int*>(w);
    p.err = device_error_word();
    const unsigned rows = (unsigned)(a.B * (greedy ? a.K + 1 : 2 * a.K + 1));
    cudaError_t e = greedy ? launch_pdl(k_verify_stats<true>, dim3(rows * p.C), dim3(kThreads), 0, st, p)
                           : launch_pdl(k_verify_stats<false>, dim3(rows * p.C), dim3(kThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    return greedy ? launch_pdl(k_verify_greedy, dim3((a.B + 7) / 8), dim3(kThreads), 0, st, p)
                  : launch_pdl(k_verify_race, dim3((unsigned)(a.B * p.C)), dim3(kThreads), 0, st, p);
}

}  // namespace tfm
