// k_packed.cu - causal attention over packed sequences of different lengths.
//
// o_i = sum_j p_ij v_j with p_i = softmax_j(scale q_i . k_j) over the keys of
// row i's own sequence, max(start, i - window + 1) <= j <= i (window 0: from the
// sequence's start); query head h reads kv head h / (H / Hkv).
#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

// Rows [start, start + len) of sequence b, or an empty range for offsets that
// decrease or leave [0, T].
struct SeqRange {
    int start, len;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* __restrict__ cu, int b, int T) {
    const int s = __ldg(cu + b), e = __ldg(cu + b + 1);
    const bool ok = s >= 0 && s <= e && e <= T;
    return SeqRange{ok ? s : 0, ok ? e - s : 0};
}

template <typename E>
__device__ __forceinline__ float to_f32(E x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float* d, float x) { *d = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* d, float x) { *d = __float2bfloat16_rn(x); }

struct PackedStrides {
    int64_t qt, qh, kt, kh, vt, vh, ot, oh;
};

// One warp per (row, head): lane l holds coordinates l, l + 32, ...; the visible
// keys in order with a running maximum and sum.
template <typename E>
__global__ void __launch_bounds__(256) k_packed_rows(const E* __restrict__ q, const E* __restrict__ k,
                                                     const E* __restrict__ v, E* __restrict__ o,
                                                     const int32_t* __restrict__ cu, int n_seq, int T,
                                                     int H, int Hkv, int dh, PackedStrides sd,
                                                     float scale, int window, int* err) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < n_seq; b += blockDim.x) {
            const int s = cu[b], e = cu[b + 1];
            if (s < 0 || s > e || e > T) raise_error(err, TFM_EINVAL);
        }
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (w >= (int64_t)T * H) return;
    const int i = (int)(w / H), h = (int)(w - (int64_t)i * H), g = h / (H / Hkv);
    // the last sequence that starts at or before row i
    int lo = 0, hi = n_seq;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i) lo = mid + 1; else hi = mid;
    }
    if (lo == 0) return;
    const SeqRange r = seq_range(cu, lo - 1, T);
    if (i < r.start || i >= r.start + r.len) return;
    const E* qr = q + i * sd.qt + h * sd.qh;
    float qv[4], acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int d = lane + 32 * t;
        qv[t] = d < dh ? to_f32(qr[d]) : 0.f;
        acc[t] = 0.f;
    }
    float mx = -INFINITY, sum = 0.f;
    const int j0 = (window > 0 && i - window + 1 > r.start) ? i - window + 1 : r.start;
    for (int j = j0; j <= i; ++j) {
        const E* kr = k + j * sd.kt + g * sd.kh;
        const E* vr = v + j * sd.vt + g * sd.vh;
        float part = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (lane + 32 * t < dh) part = fmaf(qv[t], to_f32(kr[lane + 32 * t]), part);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
        const float s = part * scale;
        const float mnew = fmaxf(mx, s);
        const float corr = expf(mx - mnew), p = expf(s - mnew);
        sum = sum * corr + p;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (lane + 32 * t < dh) acc[t] = acc[t] * corr + p * to_f32(vr[lane + 32 * t]);
        mx = mnew;
    }
    const float inv = 1.0f / sum;
    E* orow = o + i * sd.ot + h * sd.oh;
#pragma unroll
    for (int t = 0; t < 4; ++t)
        if (lane + 32 * t < dh) from_f32(orow + lane + 32 * t, acc[t] * inv);
}

template <typename E>
cudaError_t launch_rows(const PackedArgs& a, cudaStream_t st) {
    const int64_t blocks = ((int64_t)a.T * a.H + 7) / 8;
    const PackedStrides sd{a.strides[0], a.strides[1], a.strides[2], a.strides[3],
                           a.strides[4], a.strides[5], a.strides[6], a.strides[7]};
    return launch_pdl(k_packed_rows<E>, dim3((unsigned)blocks), dim3(256), 0, st,
                      static_cast<const E*>(a.q), static_cast<const E*>(a.k),
                      static_cast<const E*>(a.v), static_cast<E*>(a.o), a.cu, a.n_seq, a.T, a.H,
                      a.Hkv, a.dh, sd, a.scale, a.window, device_error_word());
}

}  // namespace

size_t packed_workspace_bytes(int T, int n_seq) { return 256 + 16 * ((size_t)T / 128 + n_seq); }

tfm_status launch_packed_attention(const PackedArgs& a, cudaStream_t st, cudaError_t* e) {
    *e = a.bf16 ? launch_rows<__nv_bfloat16>(a, st) : launch_rows<float>(a, st);
    return TFM_OK;
}

}  // namespace tfm
