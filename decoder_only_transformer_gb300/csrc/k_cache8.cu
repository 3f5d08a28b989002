// k_cache8.cu - writing new keys and values into the 8-bit cache, and reading them back.
//
// Write: a block of positions of one head is a unit.  With m the largest magnitude of its
// new rows and need = m / top (top = 127 or 448), the block's scale s is need if no
// earlier position of the sequence lies in it; otherwise it stays, or, if need is above it, is doubled until it
// covers need and the codes that are there are requantised: powers of two, so that a code
// is rounded at most once per doubling and the errors of all doublings together stay below
// one step (e4m3 codes only change their exponent, and lose bits only as subnormals).
// New codes are x / s, nearest, ties to even.
//
// Read: value = code * scale, rounded once.
//
// Both are bound by memory, one pass: the warps of a unit (one for 2048 elements) hold its rows in
// registers between the maximum and the codes; 16-byte loads of the rows, 8-byte stores
// of codes (a warp covers whole 32-byte sectors).  The instructions per element count too:
// magnitudes of bf16 rows are compared in pairs, as integers; a code is found by rounding x / s
// from below and from above (codes_of4).  The unit of a warp is found without a scan: block j of
// sequence b has the number cu[b] / block + 2 b + j, which leaves room for a partly filled
// block at either end.  Neighbouring warps take neighbouring heads, whose rows lie side by side
// (CTAs of 4 units where 8 fit: 20 for 15 us).
//
// Measured (graph replays): 32768 tokens of 4 x 128, bf16 and e4m3: written in 23.0 us (4.4 TB/s; issue
// slots 60 %), read back in 18.4 (5.5); from and to fp32 rows 34.9 and 37.9; 24 prompts of up to 1024 tokens of 12 x 64, int8,
// blocks of 16: 15.4 and 11.0 us (fp32: 19.2 and 19.1); one token of each of 64 sequences: 5.5 us.
#include "cache8.cuh"

namespace tfm {

namespace {

constexpr int kMaxThreads8 = 256;
static_assert(kMaxThreads8 % 256 == 0, "the up to 8 warps of a unit meet at a barrier: a CTA holds whole units");
constexpr int kAtOnce = 95;           // sequences whose offsets and lengths a warp looks at together

struct Geom8 {
    int B, T, Hkv, max_seq, nblk;
    int per;                       // rows per sequence without offsets
    int per_units;                 // units per sequence without offsets
    int shift;                     // log2(block)
    int units;                     // of a kv head's keys
    int warps;                     // of a unit
    int64_t s[4];                  // k token, k head, v token, v head
};

// Sequence of unit u, the unit's number in it, and where its rows lie: the last b with cu[b] / block + 2 b <= u.
__device__ __forceinline__ SeqRows find_seq(const int32_t* __restrict__ cu, const int32_t* __restrict__ lens, const Geom8& g,
                                            int u, int& b, int& j) {
    if (!cu) {
        b = u / g.per_units;
        j = u - b * g.per_units;
        return seq_rows(cu, lens, b, g.per, g.T, g.max_seq);
    }
    // every warp for itself
    const int lane = threadIdx.x & 31;
    int lo = 0;
    if (g.B > 32 && g.B <= kAtOnce) {
        // All of them at once, lengths too: one wait instead of three, in more instructions.  At once against step by step (us), a
        // token's write and read of up to 600 of 4 x 128, and prompts of 12 x 64 in blocks of 16 written and read: 24 sequences
        // 4.1 for 4.1, 6.2 for 5.5, 15.8 for 15.3, 11.7 for 11.0; 48: 4.8 for 4.8, 10.3 for 10.9, 15.7 for 16.4, 11.6 for 11.7;
        // 64: 5.5 for 5.5, 13.0 for 13.4, 14.6 for 15.1, 11.0 for 11.0; 95: 6.9 for 6.9, 17.9 for 18.5, 14.3 for 14.4, 10.3 for
        // 10.3; with a fourth word of a lane, 96: 7.5 for 6.9, 18.5 for 18.7, 14.4 for 14.4, 11.0 for 10.3; 127: 8.3 for 8.3, 24.0
        // for 24.2, 15.3 for 15.1, 11.7 for 11.0.
        constexpr int N = (kAtOnce + 1) / 32;
        int a[N], len[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] = __ldg(cu + min(lane + 32 * i, g.B));
            len[i] = __ldg(lens + min(lane + 32 * i, g.B - 1));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = lane + 32 * i;
            const unsigned below = __ballot_sync(0xffffffffu, x < g.B && (int64_t)(a[i] >> g.shift) + 2 * x <= u);
            if (below) lo = 32 * i + 31 - __clz(below);
        }
        const auto at = [&](const int (&v)[N], int x) {
            int y = v[0];
#pragma unroll
            for (int i = 1; i < N; ++i)
                if (x >= 32 * i) y = v[i];
            return __shfl_sync(0xffffffffu, y, x & 31);
        };
        b = lo;
        const int row0 = at(a, lo);
        j = u - ((row0 >> g.shift) + 2 * lo);
        return seq_rows(row0, at(a, lo + 1), at(len, lo), g.T, g.max_seq);
    }
    // 32 places at a time
    int n = g.B;                                           // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int x = lo + lane * step;
        const bool below = lane * step < n && (int64_t)(__ldg(cu + x) >> g.shift) + 2 * x <= u;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
        const int rest = n - last * step;
        lo += last * step;
        n = rest < step ? rest : step;
    }
    b = lo;
    j = u - ((__ldg(cu + lo) >> g.shift) + 2 * lo);
    return seq_rows(cu, lens, lo, g.per, g.T, g.max_seq);
}

// Every sequence's rows and length are looked at once, by one CTA.
__device__ __forceinline__ void check_rows(const int32_t* __restrict__ cu, const int32_t* __restrict__ lens,
                                           const Geom8& g, int* err) {
    bool bad = false;
    for (int b = threadIdx.x; b < g.B; b += blockDim.x) {
        const SeqRows s = seq_rows(cu, lens, b, g.per, g.T, g.max_seq);
        bad = bad || !s.ok || s.n > s.len;
    }
    if (bad) raise_error(err, TFM_EINVAL);
}

// NVEC vectors of 8 elements of a unit's rows.  (Rows, codes and scales are read past the L1 cache: a
// launch that overlaps the end of the one before may share an SM with its reads of lines that other SMs went on to
// write.)
template <typename T, int NVEC>
struct Rows8;
template <int NVEC>
struct Rows8<__nv_bfloat16, NVEC> {
    uint4 w[NVEC];
    __device__ __forceinline__ void clear(int i) { w[i] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(int i, const __nv_bfloat16* p) { w[i] = __ldcg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(int i, float* x) const {
        x[0] = bf16_lo(w[i].x), x[1] = bf16_hi(w[i].x), x[2] = bf16_lo(w[i].y), x[3] = bf16_hi(w[i].y);
        x[4] = bf16_lo(w[i].z), x[5] = bf16_hi(w[i].z), x[6] = bf16_lo(w[i].w), x[7] = bf16_hi(w[i].w);
    }
    // the largest magnitude as the integer that its bits are (those that are not finite beyond all others)
    __device__ __forceinline__ float top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NVEC; ++i) {
            m = __vmaxu2(m, w[i].x & 0x7FFF7FFFu);
            m = __vmaxu2(m, w[i].y & 0x7FFF7FFFu);
            m = __vmaxu2(m, w[i].z & 0x7FFF7FFFu);
            m = __vmaxu2(m, w[i].w & 0x7FFF7FFFu);
        }
        return __uint_as_float(max(m >> 16, m & 0xFFFFu) << 16);
    }
};
template <int NVEC>
struct Rows8<float, NVEC> {
    uint4 w[2 * NVEC];
    __device__ __forceinline__ void clear(int i) { w[2 * i] = w[2 * i + 1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(int i, const float* p) {
        w[2 * i] = __ldcg(reinterpret_cast<const uint4*>(p));
        w[2 * i + 1] = __ldcg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void get(int i, float* x) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[4 * j] = __uint_as_float(w[2 * i + j].x), x[4 * j + 1] = __uint_as_float(w[2 * i + j].y);
            x[4 * j + 2] = __uint_as_float(w[2 * i + j].z), x[4 * j + 3] = __uint_as_float(w[2 * i + j].w);
        }
    }
    __device__ __forceinline__ float top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2 * NVEC; ++i) {
            m = max(max(m, w[i].x & 0x7FFFFFFFu), w[i].y & 0x7FFFFFFFu);
            m = max(max(m, w[i].z & 0x7FFFFFFFu), w[i].w & 0x7FFFFFFFu);
        }
        return __uint_as_float(m);
    }
};

// A warp's unit: block `blk` of positions [p0, p0 + block) of kv head h of sequence b, of which
// [lo, hi) are new; k or v.
struct Unit {
    int h, isv, b, blk, p0, lo, hi;
    int64_t row0;                  // row of position 0 (positions before the new ones have none)
    bool live;
};
__device__ __forceinline__ Unit find_unit(const int32_t* __restrict__ cu, const int32_t* __restrict__ lens, const Geom8& g,
                                          int64_t flat) {
    Unit n;
    const int per = 2 * g.Hkv;                             // k's heads, then v's
    const int u = (int)(flat / per), x = (int)(flat - (int64_t)u * per);
    n.isv = x >= g.Hkv;
    n.h = n.isv ? x - g.Hkv : x;
    n.live = u < g.units;
    if (!n.live) return n;
    int j;
    const SeqRows s = find_seq(cu, lens, g, u, n.b, j);
    const int start = s.len - s.n;
    n.blk = (start >> g.shift) + j;
    n.live = s.ok && s.n > 0 && s.n <= s.len && j >= 0 && n.blk <= ((s.len - 1) >> g.shift);
    n.p0 = n.blk << g.shift;
    n.lo = max(n.p0, start);
    n.hi = min(n.p0 + (1 << g.shift), s.len);
    n.row0 = (int64_t)s.row0 - start;
    return n;
}

// W warps of a unit (g.warps of them) hold NVEC vectors of 8 elements a thread.
template <typename T, bool E4M3, int DH, int NVEC>
__global__ void __launch_bounds__(kMaxThreads8)
    k_cache8_write(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                   float* __restrict__ ks, float* __restrict__ vs, const int32_t* __restrict__ cu,
                   const int32_t* __restrict__ lens, const Geom8 g, int* err) {
    constexpr int kVR = DH / 8;                            // vectors of a row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / g.warps, tid = threadIdx.x - slot * g.warps * 32, threads = g.warps * 32;
    __shared__ float warp_top[2][kMaxThreads8 / 32];       // of the first look at a unit, of a second
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) check_rows(cu, lens, g, err);
    // Every warp finds the unit for itself.  All warps of a unit come to its barriers, whatever they have read of lengths
    // that something changes meanwhile.
    Unit n = find_unit(cu, lens, g, (int64_t)blockIdx.x * (kMaxThreads8 / threads) + slot);
    if (!n.live) {
        if (g.warps == 1) return;
        n.isv = n.h = n.b = n.blk = n.p0 = n.lo = n.hi = 0;
        n.row0 = 0;
    }
    // vector i of this thread: position first + i step, the same columns
    const int first = n.p0 + tid / kVR, step = threads / kVR;
    const unsigned count = n.hi - n.lo;                    // new positions
    const int64_t st = g.s[n.isv ? 2 : 0], bh = (int64_t)n.b * g.Hkv + n.h;
    const T* src = (n.isv ? v : k) + (int64_t)n.h * g.s[n.isv ? 3 : 1] + (n.row0 + first) * st + tid % kVR * 8;
    uint8_t* codes = (n.isv ? vc : kc) + (bh * g.max_seq + n.p0) * DH;
    float* scale = (n.isv ? vs : ks) + bh * g.nblk + n.blk;

    Rows8<T, NVEC> x;
    const int64_t ahead = step * st;
#pragma unroll
    for (int i = 0; i < NVEC; ++i, src += ahead) {
        if ((unsigned)(first + i * step - n.lo) < count) x.load(i, src);
        else x.clear(i);
    }
    const bool held = n.lo > n.p0;                         // earlier positions of the sequence lie in the block
    const float old = held ? __ldcg(scale) : 0.0f;
    const auto unit_max = [&](float y, int look) {
#pragma unroll
        for (int o = 16; o; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
        if (g.warps > 1) {
            if (lane == 0) warp_top[look][warp] = y;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(threads) : "memory");
            for (int w = 0; w < g.warps; ++w) y = fmaxf(y, warp_top[look][slot * g.warps + w]);
        }
        return y;
    };
    // (a NaN is passed on as an infinity: fmaxf would drop it)
    float top = x.top();
    top = unit_max(top < INFINITY ? top : INFINITY, 0);
    const bool odd = !(top < INFINITY);                    // something is not finite: the largest that is
    if (odd) {
        if (tid == 0) raise_error(err, TFM_EINVAL);
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < NVEC; ++i) {
            float f[8];
            x.get(i, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (fabsf(f[e]) < INFINITY) top = fmaxf(top, fabsf(f[e]));
        }
        top = unit_max(top, 1);
    }
    if (!n.live) return;
    const float need = top > 0.0f ? fmaxf(__fdiv_rn(top, code_top<E4M3>()), 0x1p-126f) : 0.0f;
    float sc = old > 0.0f ? old : need;
    int up = 0;
    if (need > sc) {                                       // old > 0 here
        up = ilogbf(need) - ilogbf(sc);
        sc = ldexpf(old, up);
        if (sc < need) sc = ldexpf(old, ++up);
    }
    if (!(sc > 0.0f)) sc = 0.0f;
    if (up) {
        const float down = ldexpf(1.0f, -up);
        for (int e = tid; e < (n.lo - n.p0) * kVR; e += threads) {
            uint2* at = reinterpret_cast<uint2*>(codes) + e;
            const uint2 w = __ldcg(at);
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = code_value<E4M3>((i < 4 ? w.x : w.y) >> (8 * (i & 3))) * down;
                c[i >> 2] |= code_of<E4M3>(y) << (8 * (i & 3));
            }
            *at = make_uint2(c[0], c[1]);
        }
    }
    const bool plain = !odd && sc >= 0x1p-100f && sc <= 0x1p100f;
    const Recip rc = recip<E4M3>(plain ? sc : 1.0f, sizeof(T) == 2);
    const auto store = [&](auto code8) {
#pragma unroll
        for (int i = 0; i < NVEC; ++i) {
            if ((unsigned)(first + i * step - n.lo) >= count) continue;
            float f[8];
            x.get(i, f);
            reinterpret_cast<uint2*>(codes)[tid + i * threads] = code8(f);
        }
    };
    if (sizeof(T) == 2 && plain && rc.sure) {
        store([&](const float* f) { return make_uint2(codes_of4<E4M3, true>(f, rc), codes_of4<E4M3, true>(f + 4, rc)); });
    } else if (plain) {
        store([&](const float* f) { return make_uint2(codes_of4<E4M3, false>(f, rc), codes_of4<E4M3, false>(f + 4, rc)); });
    } else {
        store([&](const float* f) {
            uint32_t w[2] = {0, 0};
            if (sc > 0.0f)
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j >> 2] |= code_exact<E4M3>(f[j], sc) << (8 * (j & 3));
            return make_uint2(w[0], w[1]);
        });
    }
    if (tid == 0) *scale = sc;
}

// The values of 8 codes.
template <bool E4M3>
__device__ __forceinline__ void values8(uint2 w, float sc, float* f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = h ? w.y : w.x;
        if constexpr (E4M3) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(i ? c >> 16 : c & 0xFFFFu), __NV_E4M3);
                const float2 z = __half22float2(__half2(y));
                f[4 * h + 2 * i] = z.x * sc;
                f[4 * h + 2 * i + 1] = z.y * sc;
            }
        } else {
            // the byte, its sign bit turned over, as the last one of 2^23 + (c + 128)
            const uint32_t b = c ^ 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * h + i] = (__uint_as_float(__byte_perm(b, 0x4B000000u, 0x7440 + i)) - 8388736.0f) * sc;
        }
    }
}

// (Four CTAs an SM for 2048 elements a warp: with five or six the last ones lie on some SMs only, 64 chats of up
// to 600 x 4 x 128 15.7 and 14.3 for 13.6 us, 16 of up to 1000 6.2 and 6.9 for 5.5; with three too little is on
// its way, 15.0 and 7.5.)
template <typename T, bool E4M3, int DH, int NVEC>
__global__ void __launch_bounds__(kMaxThreads8, 4)
    k_cache8_read(T* __restrict__ k, T* __restrict__ v, const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                  const float* __restrict__ ks, const float* __restrict__ vs, const int32_t* __restrict__ cu,
                  const int32_t* __restrict__ lens, const Geom8 g, int* err) {
    constexpr int kVR = DH / 8;
    const int slot = (threadIdx.x >> 5) / g.warps, tid = threadIdx.x - slot * g.warps * 32, threads = g.warps * 32;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) check_rows(cu, lens, g, err);
    const Unit n = find_unit(cu, lens, g, (int64_t)blockIdx.x * (kMaxThreads8 / threads) + slot);
    if (!n.live) return;
    const int first = n.p0 + tid / kVR, step = threads / kVR;
    const unsigned count = n.hi - n.lo;
    const int64_t st = g.s[n.isv ? 2 : 0], bh = (int64_t)n.b * g.Hkv + n.h;
    T* at = (n.isv ? v : k) + (int64_t)n.h * g.s[n.isv ? 3 : 1] + (n.row0 + first) * st + tid % kVR * 8;
    const uint2* codes = reinterpret_cast<const uint2*>((n.isv ? vc : kc) + (bh * g.max_seq + n.p0) * DH);
    const float sc = __ldcg((n.isv ? vs : ks) + bh * g.nblk + n.blk);
    uint2 w[NVEC];
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        if ((unsigned)(first + i * step - n.lo) < count) w[i] = __ldcg(codes + tid + i * threads);
    }
    const int64_t ahead = step * st;
#pragma unroll
    for (int i = 0; i < NVEC; ++i, at += ahead) {
        if ((unsigned)(first + i * step - n.lo) >= count) continue;
        float f[8];
        values8<E4M3>(w[i], sc, f);
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(at) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                       pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        } else {
            reinterpret_cast<float4*>(at)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(at)[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
}

Geom8 geom8(const Cache8Args& a) {
    Geom8 g{};
    g.B = a.B;
    g.T = a.T;
    g.Hkv = a.Hkv;
    g.max_seq = a.max_seq;
    g.shift = __builtin_ctz(a.block);
    g.nblk = (a.max_seq + a.block - 1) >> g.shift;
    g.per = a.cu ? 0 : a.T / a.B;
    g.per_units = a.cu ? 0 : (g.per + a.block - 2) / a.block + 1;      // n positions touch at most so many blocks
    g.units = a.cu ? (a.T >> g.shift) + 2 * a.B : a.B * g.per_units;
    // a warp holds up to 8 vectors a thread: 1 to 8 warps a unit
    const int vecs = a.block * a.dh / 8;
    g.warps = vecs > 256 ? vecs / 256 : 1;
    for (int i = 0; i < 4; ++i) g.s[i] = a.strides[i];
    return g;
}

template <bool READ, typename T, bool E4M3, int DH, int NVEC>
cudaError_t launch8(const Cache8Args& a, cudaStream_t st) {
    const Geom8 g = geom8(a);
    const int per_cta = kMaxThreads8 / (32 * g.warps);
    const unsigned ctas = (unsigned)(((int64_t)g.units * 2 * a.Hkv + per_cta - 1) / per_cta);
    if constexpr (READ)
        return launch_pdl(k_cache8_read<T, E4M3, DH, NVEC>, dim3(ctas), dim3(kMaxThreads8), 0, st,
                          static_cast<T*>(const_cast<void*>(a.k)), static_cast<T*>(const_cast<void*>(a.v)), a.kc, a.vc, a.ks,
                          a.vs, a.cu, a.lens, g, device_error_word());
    else
        return launch_pdl(k_cache8_write<T, E4M3, DH, NVEC>, dim3(ctas), dim3(kMaxThreads8), 0, st,
                          static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.kc, a.vc, a.ks, a.vs, a.cu, a.lens, g,
                          device_error_word());
}

template <bool READ, typename T, bool E4M3>
cudaError_t by_dh(const Cache8Args& a, cudaStream_t st) {
    const int vecs = a.block * a.dh / 8;
    if (a.dh == 32) return vecs == 64 ? launch8<READ, T, E4M3, 32, 2>(a, st) : vecs == 128 ? launch8<READ, T, E4M3, 32, 4>(a, st)
                                                                                         : launch8<READ, T, E4M3, 32, 8>(a, st);
    if (a.dh == 64) return vecs == 128 ? launch8<READ, T, E4M3, 64, 4>(a, st) : launch8<READ, T, E4M3, 64, 8>(a, st);
    return launch8<READ, T, E4M3, 128, 8>(a, st);
}

template <bool READ>
cudaError_t by_type(const Cache8Args& a, cudaStream_t st) {
    if (a.bf16) return a.e4m3 ? by_dh<READ, __nv_bfloat16, true>(a, st) : by_dh<READ, __nv_bfloat16, false>(a, st);
    return a.e4m3 ? by_dh<READ, float, true>(a, st) : by_dh<READ, float, false>(a, st);
}

}  // namespace

cudaError_t launch_cache8_write(const Cache8Args& a, cudaStream_t st) { return by_type<false>(a, st); }
cudaError_t launch_cache8_read(const Cache8Args& a, cudaStream_t st) { return by_type<true>(a, st); }

}  // namespace tfm
