// k_cache8_attn.cu - attention of the newest tokens of every sequence over its 8-bit cache.
//
// Row (sequence b, new token t of n, head h), at position p = len - n + t:
//   o = sum_j w_j s_v(j) c_v(j) / sum_j w_j,  w_j = exp(scale s_k(j) q . c_k(j) - max)
// over the positions max(0, p - window + 1) <= j <= p of kv head h / (H / Hkv); s_k, s_v are
// the scales of j's block.  A row that sees nothing is zero.
//
// One CTA per row, a warp per key: scores by a sum over the lanes, a running maximum and
// sum per warp, joined at the end.
#include "cache8.cuh"

namespace tfm {

namespace {

constexpr int kSimpleWarps = 8;

template <bool E4M3, int DH>
__global__ void __launch_bounds__(kSimpleWarps * 32)
    k_cache8_rows(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ kc, const uint8_t* __restrict__ vc,
                  const float* __restrict__ ks, const float* __restrict__ vs, __nv_bfloat16* __restrict__ o,
                  const int32_t* __restrict__ cu, const int32_t* __restrict__ lens, const Cache8AttnArgs a, int* err) {
    constexpr int E = DH / 32;
    __shared__ float acc[kSimpleWarps][DH];
    __shared__ float2 ml[kSimpleWarps];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    SeqRows s = seq_rows(cu, lens, b, cu ? 0 : a.T / a.B, a.T, a.max_seq);
    if (s.n > a.max_new) s.ok = false, s.n = 0;
    if (!s.ok) {
        if (threadIdx.x == 0) raise_error(err, TFM_EINVAL);
        s.len = 0;
    }
    if (t >= s.n) return;
    const int p = s.len - s.n + t;
    const int first = a.window > 0 ? max(0, p - a.window + 1) : 0;
    const int64_t row = s.row0 + t, bh = (int64_t)b * a.Hkv + h / (a.H / a.Hkv);
    const int nblk = (a.max_seq + a.block - 1) / a.block;
    float x[E], sum[E], m = -INFINITY, l = 0.0f;
    for (int i = 0; i < E; ++i) {
        x[i] = __bfloat162float(q[row * a.strides[0] + h * a.strides[1] + lane * E + i]) * a.scale * 1.4426950408889634f;
        sum[i] = 0.0f;
    }
    for (int j = first + warp; j <= p; j += kSimpleWarps) {
        const uint8_t* kr = kc + (bh * a.max_seq + j) * DH + lane * E;
        const uint8_t* vr = vc + (bh * a.max_seq + j) * DH + lane * E;
        float d = 0.0f;
        for (int i = 0; i < E; ++i) d += x[i] * code_value<E4M3>(kr[i]);
        for (int w = 16; w; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
        d *= ks[bh * nblk + j / a.block];
        const float nm = fmaxf(m, d), keep = m == -INFINITY ? 0.0f : exp2f(m - nm), e = exp2f(d - nm);
        const float ev = e * vs[bh * nblk + j / a.block];
        for (int i = 0; i < E; ++i) sum[i] = sum[i] * keep + ev * code_value<E4M3>(vr[i]);
        l = l * keep + e;
        m = nm;
    }
    for (int i = 0; i < E; ++i) acc[warp][lane * E + i] = sum[i];
    if (lane == 0) ml[warp] = make_float2(m, l);
    __syncthreads();
    if (threadIdx.x >= DH) return;
    float top = -INFINITY, tl = 0.0f, v = 0.0f;
    for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, ml[w].x);
    for (int w = 0; w < kSimpleWarps; ++w) {
        const float f = ml[w].x == -INFINITY ? 0.0f : exp2f(ml[w].x - top);
        tl += f * ml[w].y;
        v += f * acc[w][threadIdx.x];
    }
    o[row * a.strides[2] + h * a.strides[3] + threadIdx.x] = __float2bfloat16_rn(first <= p ? v / tl : 0.0f);
}

template <bool E4M3>
cudaError_t launch_rows(const Cache8AttnArgs& a, cudaStream_t st) {
    const dim3 grid(a.H, a.max_new, a.B);
    auto go = [&](auto kernel) {
        kernel<<<grid, kSimpleWarps * 32, 0, st>>>(static_cast<const __nv_bfloat16*>(a.q), a.kc, a.vc, a.ks, a.vs,
                                                   static_cast<__nv_bfloat16*>(a.o), a.cu, a.lens, a, device_error_word());
        return cudaGetLastError();
    };
    switch (a.dh) {
        case 32: return go(k_cache8_rows<E4M3, 32>);
        case 64: return go(k_cache8_rows<E4M3, 64>);
        default: return go(k_cache8_rows<E4M3, 128>);
    }
}

}  // namespace

size_t cache8_attention_workspace_bytes(int B, int H, int Hkv, int max_new, int dh) {
    (void)B, (void)H, (void)Hkv, (void)max_new, (void)dh;
    return 16;
}

tfm_status launch_cache8_attention(const Cache8AttnArgs& a, cudaStream_t st, cudaError_t* e) {
    *e = a.e4m3 ? launch_rows<true>(a, st) : launch_rows<false>(a, st);
    return TFM_OK;
}

}  // namespace tfm
