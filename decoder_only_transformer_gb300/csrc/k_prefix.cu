// k_prefix.cu - attention of the newest T tokens of every sequence over a
// prefix the whole batch shares and each sequence's own cache.
//
// Row (b, h, t): o = sum_j p_j v_j, p = softmax(scale q . k_j) over the keys
// [0, P) of the prefix and the own keys [0, lens[b] - (T - 1 - t)).
#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

// One warp per row.
__global__ void __launch_bounds__(256) k_prefix_rows(
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kp,
    const __nv_bfloat16* __restrict__ vp, const __nv_bfloat16* __restrict__ kc,
    const __nv_bfloat16* __restrict__ vc, __nv_bfloat16* __restrict__ o,
    const int32_t* __restrict__ lens, int B, int H, int Hkv, int T, int P, int max_prefix,
    int max_seq, int dh, float scale, int* err) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int w = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= B * H * T) return;
    const int b = w / (H * T), h = (w / T) % H, t = w % T, g = h / (H / Hkv);
    int len = lens[b];
    if (len < 0 || len > max_seq) {
        len = 0;
        raise_error(err, TFM_EINVAL);
    }
    const int own = max(0, len - (T - 1 - t));
    const __nv_bfloat16* qr = q + (int64_t)w * dh;
    float qv[4], acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        qv[c] = lane + 32 * c < dh ? __bfloat162float(qr[lane + 32 * c]) : 0.f;
        acc[c] = 0.f;
    }
    float mx = -INFINITY, sum = 0.f;
    for (int j = 0; j < P + own; ++j) {
        const bool pre = j < P;
        const int64_t row = pre ? (int64_t)g * max_prefix + j : ((int64_t)b * Hkv + g) * max_seq + (j - P);
        const __nv_bfloat16* kr = (pre ? kp : kc) + row * dh;
        const __nv_bfloat16* vr = (pre ? vp : vc) + row * dh;
        float part = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (lane + 32 * c < dh) part = fmaf(qv[c], __bfloat162float(kr[lane + 32 * c]), part);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
        const float s = part * scale;
        const float mnew = fmaxf(mx, s);
        const float corr = expf(mx - mnew), p = expf(s - mnew);
        sum = sum * corr + p;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (lane + 32 * c < dh) acc[c] = acc[c] * corr + p * __bfloat162float(vr[lane + 32 * c]);
        mx = mnew;
    }
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;    // no key at all: zeros
    __nv_bfloat16* orow = o + ((int64_t)(b * T + t) * H + h) * dh;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (lane + 32 * c < dh) orow[lane + 32 * c] = __float2bfloat16_rn(acc[c] * inv);
}

}  // namespace

size_t prefix_workspace_bytes(int B, int H, int Hkv, int T, int dh) { return 256; }

tfm_status launch_prefix_attention(const PrefixArgs& a, cudaStream_t st, cudaError_t* e) {
    using bf = __nv_bfloat16;
    *e = launch_pdl(k_prefix_rows, dim3((unsigned)((a.B * a.H * a.T + 7) / 8)), dim3(256), 0, st,
                    static_cast<const bf*>(a.q), static_cast<const bf*>(a.kp),
                    static_cast<const bf*>(a.vp), static_cast<const bf*>(a.kc),
                    static_cast<const bf*>(a.vc), static_cast<bf*>(a.o), a.lens, a.B, a.H, a.Hkv,
                    a.T, a.P, a.max_prefix, a.max_seq, a.dh, a.scale, device_error_word());
    return TFM_OK;
}

}  // namespace tfm
