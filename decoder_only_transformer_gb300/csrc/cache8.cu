// cache8.cu - entry points of the 8-bit cache's operators (include/tfm.h): rotary
// positions of packed rows and their frequencies, the cache written, read and attended to.
// Argument checks only; the kernels are in k_rope_rows.cu, k_cache8.cu and k_cache8_attn.cu.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "internal.h"

namespace {

tfm_status fail(tfm_status s, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    tfm::set_last_error(buf);
    return s;
}

tfm_status cuda_fail(cudaError_t e, const char* what) {
    return fail(TFM_ECUDA, "%s: %s", what, tfm::cuda_error_text(e));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Token and head strides, in elements, of rows [T, heads, dh]: NULL is dense, and so is the
// stride of a dimension of size one and are both of no heads, which are never used.  `multiple` in bytes.
tfm_status take_strides(int64_t* out, const int64_t* strides, int n, const char* const* names, const int* heads, int64_t T,
                        int dh, int es, int multiple) {
    for (int i = 0; i < n; ++i) {
        const bool head = i & 1;
        const int64_t dense = head ? dh : (int64_t)heads[i / 2] * dh;
        if (!strides || (head ? heads[i / 2] : T) <= 1 || heads[i / 2] == 0) {
            out[i] = dense;
            continue;
        }
        const int64_t s = strides[i];
        if (s < dh || s >= ((int64_t)1 << 39) / es || s * es % multiple)
            return fail(TFM_EINVAL, "%s %s stride %lld: at least dh, a multiple of %d bytes, below 2^39 bytes", names[i / 2],
                        head ? "head" : "token", (long long)s, multiple);
        out[i] = s;
    }
    return TFM_OK;
}

constexpr int32_t kMaxPositions = 0x7fffffff - 255;

// What the three cache calls have in common.
tfm_status check_cache(int32_t B, int32_t T, int32_t Hkv, int32_t max_seq, int32_t dh, int32_t block, int32_t codes,
                       bool offsets) {
    if (B < 0 || B > 4096 || T < 0 || T > (1 << 30)) return fail(TFM_EINVAL, "B=%d outside [0, 4096] or T=%d outside [0, 2^30]", B, T);
    if (Hkv < 1 || Hkv > 4096) return fail(TFM_EINVAL, "Hkv=%d outside [1, 4096]", Hkv);
    // (positions are ints, and so are the ends of the blocks and tiles that reach beyond the last one)
    if (max_seq < 1 || max_seq > kMaxPositions || (int64_t)B * Hkv * max_seq >= (int64_t)1 << 31)
        return fail(TFM_EINVAL, "max_seq must be in [1, 2^31 - 256] and B*Hkv*max_seq below 2^31");
    if (!offsets && B && T % B) return fail(TFM_EINVAL, "without offsets T=%d must be a multiple of B=%d", T, B);
    if (codes != TFM_CODE_INT8 && codes != TFM_CODE_E4M3) return fail(TFM_EINVAL, "bad code type");
    if (dh < 1 || block < 1) return fail(TFM_EINVAL, "dh and block must be positive");
    if (dh != 32 && dh != 64 && dh != 128) return fail(TFM_EUNSUPPORTED, "8-bit cache: dh in {32, 64, 128}");
    if (block != 16 && block != 32 && block != 64 && block != 128)
        return fail(TFM_EUNSUPPORTED, "8-bit cache: blocks of 16, 32, 64 or 128 positions");
    return TFM_OK;
}

tfm_status cache_call(bool read, const void* k, const void* v, void* k_codes, void* v_codes, float* k_scales,
                      float* v_scales, const int32_t* cu_seqlens, const int32_t* lens, int32_t B, int32_t T, int32_t Hkv,
                      int32_t dh, int32_t max_seq, int32_t block, const int64_t* strides, int32_t codes, int32_t mode,
                      void* stream) {
    tfm_status st = check_cache(B, T, Hkv, max_seq, dh, block, codes, cu_seqlens != nullptr);
    if (st != TFM_OK) return st;
    if (mode != TFM_FP32 && mode != TFM_BF16) return fail(TFM_EINVAL, "bad mode");
    if (((int64_t)T / block + 2 * B) * 2 * Hkv >= (int64_t)1 << 31)
        return fail(TFM_EINVAL, "(T / block + 2 B) * 2 Hkv must be below 2^31");
    tfm::Cache8Args a{};
    static const char* const names[2] = {"k", "v"};
    const int heads[2] = {Hkv, Hkv};
    st = take_strides(a.strides, strides, 4, names, heads, T, dh, mode == TFM_BF16 ? 2 : 4, 16);
    if (st != TFM_OK) return st;
    if (B == 0 || T == 0) return TFM_OK;
    if (!k || !v || !k_codes || !v_codes || !k_scales || !v_scales || !lens) return fail(TFM_EINVAL, "NULL pointer");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16))
        return fail(TFM_EINVAL, "k, v and the codes must be 16-byte aligned");
    if (!aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(lens, 4) || !aligned(cu_seqlens, 4))
        return fail(TFM_EINVAL, "scales, lens and cu_seqlens must be 4-byte aligned");
    if (!tfm::device_error_word()) return fail(TFM_ECUDA, "device error word unavailable");
    a.k = k;
    a.v = v;
    a.kc = static_cast<uint8_t*>(k_codes);
    a.vc = static_cast<uint8_t*>(v_codes);
    a.ks = k_scales;
    a.vs = v_scales;
    a.cu = cu_seqlens;
    a.lens = lens;
    a.B = B;
    a.T = T;
    a.Hkv = Hkv;
    a.dh = dh;
    a.max_seq = max_seq;
    a.block = block;
    a.e4m3 = codes == TFM_CODE_E4M3;
    a.bf16 = mode == TFM_BF16;
    const cudaError_t e = read ? tfm::launch_cache8_read(a, static_cast<cudaStream_t>(stream))
                               : tfm::launch_cache8_write(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TFM_OK : cuda_fail(e, read ? "cache read launch" : "cache write launch");
}

bool attn_sizes_ok(int32_t B, int32_t H, int32_t Hkv, int32_t max_new) {
    return B >= 0 && B <= 4096 && H >= 1 && Hkv >= 1 && Hkv <= 4096 && H % Hkv == 0 && max_new >= 1 &&
           (int64_t)B * H * max_new <= (1 << 24);
}

}  // namespace

extern "C" {

tfm_status tfm_rope_frequencies(double theta, int32_t rot, int32_t scaling, double factor, double original, double low,
                                double high, double* inv_freq, float* mscale) {
    const double kTurn = 6.283185307179586476925;
    if (rot < 2 || rot % 2 || rot > 256) return fail(TFM_EINVAL, "rot must be even, in [2, 256]");
    if (!(theta > 1.0) || !std::isfinite(theta)) return fail(TFM_EINVAL, "theta must be > 1");
    if (scaling < TFM_ROPE_PLAIN || scaling > TFM_ROPE_WAVELENGTH) return fail(TFM_EINVAL, "unknown scaling");
    if (scaling != TFM_ROPE_PLAIN && !(factor >= 1.0 && factor <= 1e6)) return fail(TFM_EINVAL, "factor must be in [1, 1e6]");
    const bool parts = scaling == TFM_ROPE_YARN || scaling == TFM_ROPE_WAVELENGTH;
    if (parts && !(original >= 1.0 && original <= 1e9 && low > 0.0 && high > low && high <= 1e9))
        return fail(TFM_EINVAL, "original must be in [1, 1e9] and 0 < low < high <= 1e9");
    if (!inv_freq || !mscale) return fail(TFM_EINVAL, "NULL pointer");
    // Longer contexts by a larger base: the slowest pair, number rot/2 - 1, slows down by `factor`.
    const double base = scaling == TFM_ROPE_NTK && rot > 2 ? theta * std::pow(factor, rot / (rot - 2.0)) : theta;
    // The (fractional) number of the pair that turns `turns` times over the original context.
    const auto pair_of = [&](double turns) { return rot * std::log(original / (turns * kTurn)) / (2.0 * std::log(theta)); };
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == TFM_ROPE_LINEAR) f /= factor;
        if (parts) {
            double keep;                      // 1: as it is, 0: slowed down by `factor`
            if (scaling == TFM_ROPE_YARN) {
                const double lo = std::fmax(std::floor(pair_of(high)), 0.0), hi = std::fmin(std::ceil(pair_of(low)), rot - 1.0);
                keep = 1.0 - std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            } else {
                keep = std::fmin(std::fmax((original * f / kTurn - low) / (high - low), 0.0), 1.0);
            }
            f = keep * f + (1.0 - keep) * f / factor;
        }
        inv_freq[i] = f;
    }
    *mscale = scaling == TFM_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return TFM_OK;
}

tfm_status tfm_rope_rows(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                         const double* inv_freq, int32_t T, int32_t H, int32_t Hkv, int32_t dh, int32_t rot,
                         int32_t interleaved, const int64_t* strides, float mscale, int32_t mode, void* stream) {
    if (T < 0 || T > (1 << 30)) return fail(TFM_EINVAL, "T=%d outside [0, 2^30]", T);
    if (H < 1 || Hkv < 0 || H > 4096 || Hkv > 4096) return fail(TFM_EINVAL, "H in [1, 4096] and Hkv in [0, 4096] are required");
    if (dh < 2 || dh > 256) return fail(TFM_EINVAL, "dh=%d outside [2, 256]", dh);
    if (rot < 2 || rot % 2 || rot > dh) return fail(TFM_EINVAL, "rot must be even, in [2, dh]");
    if (mode != TFM_FP32 && mode != TFM_BF16) return fail(TFM_EINVAL, "bad mode");
    if (!std::isfinite(mscale)) return fail(TFM_EINVAL, "mscale must be finite");
    const int es = mode == TFM_BF16 ? 2 : 4;
    tfm::RopeRowsArgs a{};
    static const char* const names[4] = {"q", "k", "q_out", "k_out"};
    const int heads[4] = {H, Hkv, H, Hkv};
    const tfm_status st = take_strides(a.strides, strides, 8, names, heads, T, dh, es, es);
    if (st != TFM_OK) return st;
    if (T == 0) return TFM_OK;
    if (!q || !q_out || (Hkv && (!k || !k_out)) || !positions || !inv_freq) return fail(TFM_EINVAL, "NULL pointer");
    if (!aligned(q, es) || !aligned(q_out, es) || (Hkv && (!aligned(k, es) || !aligned(k_out, es))) || !aligned(positions, 4) ||
        !aligned(inv_freq, 8))
        return fail(TFM_EINVAL, "rows must be aligned to their element size, positions to 4 bytes, inv_freq to 8");
    for (int i = 0; i < 2; ++i)
        if ((i ? Hkv && k == k_out : q == q_out) && (a.strides[2 * i] != a.strides[2 * i + 4] || a.strides[2 * i + 1] != a.strides[2 * i + 5]))
            return fail(TFM_EINVAL, "%s in place: the output's strides must be the input's", names[i]);
    a.q = q;
    a.k = k;
    a.qo = q_out;
    a.ko = k_out;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.T = T;
    a.H = H;
    a.Hkv = Hkv;
    a.dh = dh;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.mscale = mscale;
    a.bf16 = mode == TFM_BF16;
    const cudaError_t e = tfm::launch_rope_rows(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TFM_OK : cuda_fail(e, "rope launch");
}

tfm_status tfm_cache8_write(const void* k, const void* v, void* k_codes, void* v_codes, float* k_scales, float* v_scales,
                            const int32_t* cu_seqlens, const int32_t* lens, int32_t B, int32_t T, int32_t Hkv, int32_t dh,
                            int32_t max_seq, int32_t block, const int64_t* strides, int32_t codes, int32_t mode,
                            void* stream) {
    return cache_call(false, k, v, k_codes, v_codes, k_scales, v_scales, cu_seqlens, lens, B, T, Hkv, dh, max_seq, block,
                      strides, codes, mode, stream);
}

tfm_status tfm_cache8_read(const void* k_codes, const void* v_codes, const float* k_scales, const float* v_scales, void* k,
                           void* v, const int32_t* cu_seqlens, const int32_t* lens, int32_t B, int32_t T, int32_t Hkv,
                           int32_t dh, int32_t max_seq, int32_t block, const int64_t* strides, int32_t codes, int32_t mode,
                           void* stream) {
    return cache_call(true, k, v, const_cast<void*>(k_codes), const_cast<void*>(v_codes), const_cast<float*>(k_scales),
                      const_cast<float*>(v_scales), cu_seqlens, lens, B, T, Hkv, dh, max_seq, block, strides, codes, mode,
                      stream);
}

size_t tfm_cache8_attention_workspace_bytes(int32_t B, int32_t H, int32_t Hkv, int32_t max_new, int32_t dh) {
    if (!attn_sizes_ok(B, H, Hkv, max_new) || (int64_t)(H / Hkv) * max_new > 128 || (dh != 32 && dh != 64 && dh != 128))
        return 0;
    return tfm::cache8_attention_workspace_bytes(B, H, Hkv, max_new, dh);
}

tfm_status tfm_cache8_attention(const void* q, const void* k_codes, const void* v_codes, const float* k_scales,
                                const float* v_scales, void* o, const int32_t* cu_seqlens, const int32_t* lens, int32_t B,
                                int32_t T, int32_t H, int32_t Hkv, int32_t max_new, int32_t dh, int32_t max_seq,
                                int32_t block, const int64_t* strides, int32_t codes, int32_t window, float scale,
                                void* workspace, size_t workspace_bytes, void* stream) {
    tfm_status st = check_cache(B, T, Hkv, max_seq, dh, block, codes, cu_seqlens != nullptr);
    if (st != TFM_OK) return st;
    if (!attn_sizes_ok(B, H, Hkv, max_new))
        return fail(TFM_EINVAL, "bad sizes: H %% Hkv == 0, max_new >= 1, B*H*max_new <= 2^24");
    if (!cu_seqlens && B && T / B > max_new) return fail(TFM_EINVAL, "max_new=%d below the T / B = %d rows of a sequence", max_new, T / B);
    if (window < 0) return fail(TFM_EINVAL, "window must be >= 0");
    // (the limit of the other attentions; the kernel itself holds scale * log2(e) as mantissa and exponent)
    if (!std::isfinite(scale) || scale > 0x1p126f) return fail(TFM_EINVAL, "scale must be finite and at most 2^126");
    if ((int64_t)(H / Hkv) * max_new > 128) return fail(TFM_EUNSUPPORTED, "8-bit cache attention: (H / Hkv) * max_new <= 128");
    tfm::Cache8AttnArgs a{};
    static const char* const names[2] = {"q", "o"};
    const int heads[2] = {H, H};
    st = take_strides(a.strides, strides, 4, names, heads, T, dh, 2, 16);
    if (st != TFM_OK) return st;
    if (B == 0 || T == 0) return TFM_OK;
    if (!q || !k_codes || !v_codes || !k_scales || !v_scales || !o || !lens || !workspace) return fail(TFM_EINVAL, "NULL pointer");
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(workspace, 16))
        return fail(TFM_EINVAL, "q, o, the codes and workspace must be 16-byte aligned");
    if (!aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(lens, 4) || !aligned(cu_seqlens, 4))
        return fail(TFM_EINVAL, "scales, lens and cu_seqlens must be 4-byte aligned");
    if (workspace_bytes < tfm::cache8_attention_workspace_bytes(B, H, Hkv, max_new, dh))
        return fail(TFM_EINVAL, "workspace too small");
    if (!tfm::device_error_word()) return fail(TFM_ECUDA, "device error word unavailable");
    a.q = q;
    a.kc = static_cast<const uint8_t*>(k_codes);
    a.vc = static_cast<const uint8_t*>(v_codes);
    a.ks = k_scales;
    a.vs = v_scales;
    a.o = o;
    a.cu = cu_seqlens;
    a.lens = lens;
    a.B = B;
    a.T = T;
    a.H = H;
    a.Hkv = Hkv;
    a.max_new = max_new;
    a.dh = dh;
    a.max_seq = max_seq;
    a.block = block;
    a.e4m3 = codes == TFM_CODE_E4M3;
    a.window = window >= max_seq ? 0 : window;       // no sequence is longer than max_seq
    a.scale = scale > 0.f ? scale : 1.0f / std::sqrt((float)dh);
    a.ws = workspace;
    cudaError_t e = cudaSuccess;
    st = tfm::launch_cache8_attention(a, static_cast<cudaStream_t>(stream), &e);
    if (st != TFM_OK) return fail(st, "could not encode the cache's tensor maps");
    return e == cudaSuccess ? TFM_OK : cuda_fail(e, "8-bit cache attention launch");
}

}  // extern "C"
