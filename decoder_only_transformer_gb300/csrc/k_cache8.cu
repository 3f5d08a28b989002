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
// Both are bound by memory, one pass: a CTA holds its unit's rows in registers between the
// maximum and the codes.  16-byte loads of the rows, 8-byte stores of codes (a warp
// covers whole 32-byte sectors).  The unit of CTA u is found without a scan: block j of
// sequence b has the number cu[b] / block + 2 b + j, which leaves room for a partly filled
// block at either end.
#include "cache8.cuh"

namespace tfm {

namespace {

constexpr int kMaxThreads8 = 256;

struct Geom8 {
    int B, T, Hkv, max_seq, nblk;
    int per;                       // rows per sequence without offsets
    int per_units;                 // units per sequence without offsets
    int shift;                     // log2(block)
    int64_t s[4];                  // k token, k head, v token, v head
};

// Sequence of unit u and the unit's number in it: the last b with cu[b] / block + 2 b <= u.
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, const Geom8& g, int u, int& j) {
    if (!cu) {
        const int b = u / g.per_units;
        j = u - b * g.per_units;
        return b;
    }
    // 32 places at a time, every warp for itself
    const int lane = threadIdx.x & 31;
    int lo = 0, n = g.B;                                   // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const bool below = lane * step < n && (int64_t)(__ldg(cu + b) >> g.shift) + 2 * b <= u;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
        const int rest = n - last * step;
        lo += last * step;
        n = rest < step ? rest : step;
    }
    j = u - ((__ldg(cu + lo) >> g.shift) + 2 * lo);
    return lo;
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

template <typename T, int NVEC>
struct Rows8;
template <int NVEC>
struct Rows8<__nv_bfloat16, NVEC> {
    uint4 w[NVEC];
    __device__ __forceinline__ void clear(int i) { w[i] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(int i, const __nv_bfloat16* p) { w[i] = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(int i, float* x) const {
        x[0] = bf16_lo(w[i].x), x[1] = bf16_hi(w[i].x), x[2] = bf16_lo(w[i].y), x[3] = bf16_hi(w[i].y);
        x[4] = bf16_lo(w[i].z), x[5] = bf16_hi(w[i].z), x[6] = bf16_lo(w[i].w), x[7] = bf16_hi(w[i].w);
    }
};
template <int NVEC>
struct Rows8<float, NVEC> {
    uint4 w[2 * NVEC];
    __device__ __forceinline__ void clear(int i) { w[2 * i] = w[2 * i + 1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(int i, const float* p) {
        w[2 * i] = __ldg(reinterpret_cast<const uint4*>(p));
        w[2 * i + 1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void get(int i, float* x) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[4 * j] = __uint_as_float(w[2 * i + j].x), x[4 * j + 1] = __uint_as_float(w[2 * i + j].y);
            x[4 * j + 2] = __uint_as_float(w[2 * i + j].z), x[4 * j + 3] = __uint_as_float(w[2 * i + j].w);
        }
    }
};

// NVEC vectors of 8 elements per thread cover a unit.
template <typename T, bool E4M3, int DH, int NVEC>
__global__ void __launch_bounds__(kMaxThreads8)
    k_cache8_write(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                   float* __restrict__ ks, float* __restrict__ vs, const int32_t* __restrict__ cu,
                   const int32_t* __restrict__ lens, const Geom8 g, int* err) {
    constexpr int kVR = DH / 8;                            // vectors of a row
    const int h = blockIdx.y, isv = blockIdx.z, tid = threadIdx.x;
    __shared__ float warp_max[kMaxThreads8 / 32];
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && h == 0 && isv == 0) check_rows(cu, lens, g, err);
    int j;
    const int b = find_seq(cu, g, blockIdx.x, j);
    const SeqRows s = seq_rows(cu, lens, b, g.per, g.T, g.max_seq);
    if (!s.ok || s.n == 0 || s.n > s.len) return;
    const int start = s.len - s.n;
    const int blk = (start >> g.shift) + j;
    if (j < 0 || blk > ((s.len - 1) >> g.shift)) return;
    const int p0 = blk << g.shift;
    const int lo = max(p0, start), hi = min(p0 + (1 << g.shift), s.len);
    const T* src = (isv ? v : k) + (int64_t)h * g.s[isv ? 3 : 1];
    const int64_t st = g.s[isv ? 2 : 0], row0 = (int64_t)s.row0 - start;
    const int64_t bh = (int64_t)b * g.Hkv + h;
    uint8_t* codes = (isv ? vc : kc) + (bh * g.max_seq + p0) * DH;
    float* scale = (isv ? vs : ks) + bh * g.nblk + blk;
    const bool held = lo > p0;                             // earlier positions of the sequence lie in the block
    const float old = held ? *scale : 0.0f;

    Rows8<T, NVEC> x;
    float top = 0.0f;
    bool odd = false;                                      // something is not finite
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        const int e = tid + i * (int)blockDim.x, p = p0 + e / kVR;
        if (p >= lo && p < hi) x.load(i, src + (row0 + p) * st + e % kVR * 8);
        else x.clear(i);
    }
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        float f[8];
        x.get(i, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = fabsf(f[e]);
            const bool fin = a < INFINITY;
            odd = odd || !fin;
            top = fmaxf(top, fin ? a : 0.0f);
        }
    }
    odd = __syncthreads_or(odd);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) warp_max[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) top = fmaxf(top, warp_max[w]);
    if (odd && tid == 0) raise_error(err, TFM_EINVAL);

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
        for (int e = tid; e < (lo - p0) * kVR; e += blockDim.x) {
            uint2* at = reinterpret_cast<uint2*>(codes) + e;
            const uint2 w = *at;
            uint32_t n[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = code_value<E4M3>((i < 4 ? w.x : w.y) >> (8 * (i & 3))) * down;
                n[i >> 2] |= code_of<E4M3>(y) << (8 * (i & 3));
            }
            *at = make_uint2(n[0], n[1]);
        }
    }
    const bool plain = !odd && sc >= 0x1p-100f && sc <= 0x1p100f;
    const float r = plain ? __frcp_rn(sc) : 0.0f;
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        const int e = tid + i * (int)blockDim.x, p = p0 + e / kVR;
        if (p < lo || p >= hi) continue;
        float f[8];
        x.get(i, f);
        bool open = !plain;
        uint2 w;
        w.x = codes4<E4M3>(f, r, open);
        w.y = codes4<E4M3>(f + 4, r, open);
        if (open) {
            uint32_t n[2] = {0, 0};
            if (plain) {
#pragma unroll
                for (int c = 0; c < 8; ++c) n[c >> 2] |= code_of<E4M3>(settled<E4M3>(f[c], sc, r)) << (8 * (c & 3));
            } else if (sc > 0.0f) {
#pragma unroll
                for (int c = 0; c < 8; ++c) n[c >> 2] |= code_exact<E4M3>(f[c], sc) << (8 * (c & 3));
            }
            w = make_uint2(n[0], n[1]);
        }
        reinterpret_cast<uint2*>(codes)[e] = w;
    }
    if (tid == 0) *scale = sc;
}

template <bool E4M3>
__device__ __forceinline__ void values8(uint2 w, float sc, float* f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = code_value<E4M3>((i < 4 ? w.x : w.y) >> (8 * (i & 3))) * sc;
}

template <typename T, bool E4M3, int DH>
__global__ void __launch_bounds__(kMaxThreads8)
    k_cache8_read(T* __restrict__ k, T* __restrict__ v, const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                  const float* __restrict__ ks, const float* __restrict__ vs, const int32_t* __restrict__ cu,
                  const int32_t* __restrict__ lens, const Geom8 g, int* err) {
    constexpr int kVR = DH / 8;
    const int h = blockIdx.y, isv = blockIdx.z, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && h == 0 && isv == 0) check_rows(cu, lens, g, err);
    int j;
    const int b = find_seq(cu, g, blockIdx.x, j);
    const SeqRows s = seq_rows(cu, lens, b, g.per, g.T, g.max_seq);
    if (!s.ok || s.n == 0 || s.n > s.len) return;
    const int start = s.len - s.n;
    const int blk = (start >> g.shift) + j;
    if (j < 0 || blk > ((s.len - 1) >> g.shift)) return;
    const int p0 = blk << g.shift;
    const int lo = max(p0, start), hi = min(p0 + (1 << g.shift), s.len);
    T* dst = (isv ? v : k) + (int64_t)h * g.s[isv ? 3 : 1];
    const int64_t st = g.s[isv ? 2 : 0], row0 = (int64_t)s.row0 - start;
    const int64_t bh = (int64_t)b * g.Hkv + h;
    const uint2* codes = reinterpret_cast<const uint2*>((isv ? vc : kc) + (bh * g.max_seq + p0) * DH);
    const float sc = __ldg((isv ? vs : ks) + bh * g.nblk + blk);
    for (int e = (lo - p0) * kVR + tid; e < (hi - p0) * kVR; e += blockDim.x) {
        const uint2 w = __ldg(codes + e);
        float f[8];
        values8<E4M3>(w, sc, f);
        T* at = dst + (row0 + p0 + e / kVR) * st + e % kVR * 8;
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
    for (int i = 0; i < 4; ++i) g.s[i] = a.strides[i];
    return g;
}

dim3 grid8(const Cache8Args& a, const Geom8& g) {
    const int64_t units = a.cu ? (int64_t)(a.T >> g.shift) + 2 * a.B : (int64_t)a.B * g.per_units;
    return dim3((unsigned)units, a.Hkv, 2);
}

template <typename T, bool E4M3, int DH>
cudaError_t write_t(const Cache8Args& a, cudaStream_t st) {
    const Geom8 g = geom8(a);
    const int vecs = a.block * DH / 8;                     // 64 .. 2048
    const int threads = vecs < kMaxThreads8 ? vecs : kMaxThreads8;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid8(a, g), dim3(threads), 0, st, static_cast<const T*>(a.k), static_cast<const T*>(a.v),
                          a.kc, a.vc, a.ks, a.vs, a.cu, a.lens, g, device_error_word());
    };
    switch (vecs / threads) {
        case 1: return go(k_cache8_write<T, E4M3, DH, 1>);
        case 2: return go(k_cache8_write<T, E4M3, DH, 2>);
        case 4: return go(k_cache8_write<T, E4M3, DH, 4>);
        default: return go(k_cache8_write<T, E4M3, DH, 8>);
    }
}

template <typename T, bool E4M3, int DH>
cudaError_t read_t(const Cache8Args& a, cudaStream_t st) {
    const Geom8 g = geom8(a);
    const int vecs = a.block * DH / 8;
    const int threads = vecs < kMaxThreads8 ? vecs : kMaxThreads8;
    return launch_pdl(k_cache8_read<T, E4M3, DH>, grid8(a, g), dim3(threads), 0, st,
                      static_cast<T*>(const_cast<void*>(a.k)), static_cast<T*>(const_cast<void*>(a.v)), a.kc, a.vc, a.ks,
                      a.vs, a.cu, a.lens, g, device_error_word());
}

template <bool READ, typename T, bool E4M3>
cudaError_t by_dh(const Cache8Args& a, cudaStream_t st) {
    switch (a.dh) {
        case 32: return READ ? read_t<T, E4M3, 32>(a, st) : write_t<T, E4M3, 32>(a, st);
        case 64: return READ ? read_t<T, E4M3, 64>(a, st) : write_t<T, E4M3, 64>(a, st);
        default: return READ ? read_t<T, E4M3, 128>(a, st) : write_t<T, E4M3, 128>(a, st);
    }
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
