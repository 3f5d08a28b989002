// batch.cu - entry points of the batched-serving operators (include/tfm.h):
// packed-prompt attention, attention over a shared prefix, verification of
// drafted tokens.  Argument checks only; the kernels are in k_packed.cu,
// k_prefix.cu and k_verify.cu.
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

// (beyond 2^126 its product with log2(e), by which the kernels scale, leaves fp32)
bool scale_ok(float scale) { return std::isfinite(scale) && scale <= 0x1p126f; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" {

size_t tfm_packed_attention_workspace_bytes(int32_t T, int32_t n_seq) {
    if (T < 0 || T > (1 << 30) || n_seq < 0 || n_seq > (1 << 20)) return 0;
    return tfm::packed_workspace_bytes(T, n_seq);
}

tfm_status tfm_packed_attention(const void* q, const void* k, const void* v, void* o,
                                const int32_t* cu_seqlens, int32_t n_seq, int32_t T, int32_t H,
                                int32_t Hkv, int32_t dh, const int64_t* strides, float scale,
                                int32_t window, int32_t mode, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (T < 0 || T > (1 << 30) || n_seq < 0 || n_seq > (1 << 20))
        return fail(TFM_EINVAL, "T=%d outside [0, 2^30] or n_seq=%d outside [0, 2^20]", T, n_seq);
    if (H < 1 || Hkv < 1 || H % Hkv) return fail(TFM_EINVAL, "bad head counts");
    if (((int64_t)T / 32 + n_seq) * H > (int64_t)1 << 30) return fail(TFM_EINVAL, "(T / 32 + n_seq) * H too large");
    if (mode != TFM_FP32 && mode != TFM_BF16) return fail(TFM_EINVAL, "bad mode");
    if (window < 0) return fail(TFM_EINVAL, "window must be >= 0");
    if (!scale_ok(scale)) return fail(TFM_EINVAL, "scale must be finite and at most 2^126");
    if (dh < 1) return fail(TFM_EINVAL, "dh must be positive");
    if (mode == TFM_BF16 && dh != 32 && dh != 64 && dh != 128)
        return fail(TFM_EUNSUPPORTED, "bf16 packed attention: dh in {32, 64, 128}");
    if (mode == TFM_FP32 && (dh % 4 || dh > 128))
        return fail(TFM_EUNSUPPORTED, "fp32 packed attention: dh %% 4 == 0, dh <= 128");
    tfm::PackedArgs a{};
    const int es = mode == TFM_BF16 ? 2 : 4;
    static const char* names[8] = {"q token", "q head", "k token", "k head",
                                   "v token", "v head", "o token", "o head"};
    for (int i = 0; i < 8; ++i) {
        const int heads = (i < 2 || i >= 6) ? H : Hkv;
        const bool head = i & 1;
        const int64_t dense = head ? dh : (int64_t)heads * dh;
        // the stride of a dimension of size one is never used
        if (!strides || (head ? heads : T) == 1) {
            a.strides[i] = dense;
            continue;
        }
        const int64_t s = strides[i];
        if (s < dh || s >= ((int64_t)1 << 39) / es || s * es % 16)
            return fail(TFM_EINVAL, "%s stride %lld: at least dh, a multiple of 16 bytes, below 2^39 bytes",
                        names[i], (long long)s);
        a.strides[i] = s;
    }
    // dense rows of an fp32 dh that is a multiple of 4, or a bf16 dh of 32 and
    // more, are multiples of 16 bytes
    if (T == 0 || n_seq == 0) return TFM_OK;
    if (!q || !k || !v || !o || !cu_seqlens || !workspace) return fail(TFM_EINVAL, "NULL pointer");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(workspace, 16))
        return fail(TFM_EINVAL, "q, k, v, o and workspace must be 16-byte aligned");
    if (!aligned(cu_seqlens, 4)) return fail(TFM_EINVAL, "cu_seqlens must be 4-byte aligned");
    if (workspace_bytes < tfm::packed_workspace_bytes(T, n_seq)) return fail(TFM_EINVAL, "workspace too small");
    if (!tfm::device_error_word()) return fail(TFM_ECUDA, "device error word unavailable");
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.cu = cu_seqlens;
    a.n_seq = n_seq;
    a.T = T;
    a.H = H;
    a.Hkv = Hkv;
    a.dh = dh;
    a.scale = scale > 0.f ? scale : 1.0f / std::sqrt((float)dh);
    a.window = window >= T ? 0 : window;             // no sequence is longer than T
    a.bf16 = mode == TFM_BF16;
    a.ws = workspace;
    cudaError_t e = cudaSuccess;
    const tfm_status st = tfm::launch_packed_attention(a, static_cast<cudaStream_t>(stream), &e);
    if (st != TFM_OK) return fail(st, "could not encode packed attention tensor maps");
    return e == cudaSuccess ? TFM_OK : cuda_fail(e, "packed attention launch");
}

static bool prefix_sizes_ok(int32_t B, int32_t H, int32_t Hkv, int32_t T) {
    return B >= 0 && B <= 4096 && H >= 1 && Hkv >= 1 && H % Hkv == 0 && T >= 1 &&
           (int64_t)B * H * T <= (1 << 24);
}

size_t tfm_prefix_attention_workspace_bytes(int32_t B, int32_t H, int32_t Hkv, int32_t T, int32_t dh) {
    if (!prefix_sizes_ok(B, H, Hkv, T) || (int64_t)(H / Hkv) * T > 128 ||
        (dh != 32 && dh != 64 && dh != 128))
        return 0;
    return tfm::prefix_workspace_bytes(B, H, Hkv, T, dh);
}

tfm_status tfm_prefix_attention(const void* q, const void* k_prefix, const void* v_prefix,
                                const void* k_cache, const void* v_cache, void* o,
                                const int32_t* lens, int32_t B, int32_t H, int32_t Hkv, int32_t T,
                                int32_t prefix_len, int32_t max_prefix, int32_t max_seq, int32_t dh,
                                float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (!prefix_sizes_ok(B, H, Hkv, T))
        return fail(TFM_EINVAL, "bad sizes: 0 <= B <= 4096, H %% Hkv == 0, T >= 1, B*H*T <= 2^24");
    if (prefix_len < 0 || max_prefix < prefix_len)
        return fail(TFM_EINVAL, "prefix_len=%d outside [0, max_prefix=%d]", prefix_len, max_prefix);
    if (max_seq < 1 || (int64_t)B * Hkv * max_seq >= (1 << 30) || (int64_t)Hkv * max_prefix > INT32_MAX)
        return fail(TFM_EINVAL, "max_seq must be positive, B*Hkv*max_seq below 2^30, Hkv*max_prefix below 2^31");
    if (!scale_ok(scale)) return fail(TFM_EINVAL, "scale must be finite and at most 2^126");
    if (dh != 32 && dh != 64 && dh != 128) return fail(TFM_EUNSUPPORTED, "prefix attention: dh in {32, 64, 128}");
    if ((int64_t)(H / Hkv) * T > 128) return fail(TFM_EUNSUPPORTED, "prefix attention: (H / Hkv) * T <= 128");
    if (tfm::prefix_key_tiles(B, H, Hkv, T, prefix_len, max_seq) > tfm::kMaxPrefixTiles)
        return fail(TFM_EINVAL, "too many key tiles: Hkv * ceil(B / floor(128 / (H / Hkv * T))) * ceil(prefix_len / 64) + "
                                "B * Hkv * ceil(max_seq / 64) at most 2^25");
    if (B == 0) return TFM_OK;
    if (!q || !k_cache || !v_cache || !o || !lens || !workspace || (prefix_len && (!k_prefix || !v_prefix)))
        return fail(TFM_EINVAL, "NULL pointer");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
        !aligned(workspace, 16) || (prefix_len && (!aligned(k_prefix, 16) || !aligned(v_prefix, 16))))
        return fail(TFM_EINVAL, "pointers must be 16-byte aligned");
    if (!aligned(lens, 4)) return fail(TFM_EINVAL, "lens must be 4-byte aligned");
    if (workspace_bytes < tfm::prefix_workspace_bytes(B, H, Hkv, T, dh)) return fail(TFM_EINVAL, "workspace too small");
    if (!tfm::device_error_word()) return fail(TFM_ECUDA, "device error word unavailable");
    tfm::PrefixArgs a{};
    a.q = q;
    a.kp = k_prefix;
    a.vp = v_prefix;
    a.kc = k_cache;
    a.vc = v_cache;
    a.o = o;
    a.lens = lens;
    a.B = B;
    a.H = H;
    a.Hkv = Hkv;
    a.T = T;
    a.P = prefix_len;
    a.max_prefix = max_prefix;
    a.max_seq = max_seq;
    a.dh = dh;
    a.scale = scale > 0.f ? scale : 1.0f / std::sqrt((float)dh);
    a.ws = workspace;
    cudaError_t e = cudaSuccess;
    const tfm_status st = tfm::launch_prefix_attention(a, static_cast<cudaStream_t>(stream), &e);
    if (st != TFM_OK) return fail(st, "could not encode prefix attention tensor maps");
    return e == cudaSuccess ? TFM_OK : cuda_fail(e, "prefix attention launch");
}

static bool verify_sizes_ok(int32_t B, int32_t K, int32_t V) {
    return B >= 0 && K >= 0 && K <= 64 && V >= 1 && V <= (1 << 24) && (int64_t)B * (K + 1) <= (1 << 20) &&
           tfm::verify_workspace_bytes(B, K, V) < (size_t)1 << 33;   // and so its grids below 2^31 CTAs
}

size_t tfm_verify_draft_workspace_bytes(int32_t B, int32_t K, int32_t V) {
    return verify_sizes_ok(B, K, V) ? tfm::verify_workspace_bytes(B, K, V) : 0;
}

tfm_status tfm_verify_draft(const float* target, int64_t ld_target, const float* draft_logits,
                            int64_t ld_draft, const int32_t* draft, const int32_t* n_draft,
                            const float* u, const float* noise, int64_t ld_noise, int32_t B,
                            int32_t K, int32_t V, float temperature, int32_t* tokens,
                            int32_t* n_accepted, void* workspace, size_t workspace_bytes,
                            void* stream) {
    if (!verify_sizes_ok(B, K, V))
        return fail(TFM_EINVAL, "bad sizes: B >= 0, 0 <= K <= 64, 1 <= V <= 2^24, B*(K+1) <= 2^20, a workspace below 2^33 bytes");
    // outside, log2(e) / temperature or a difference of logits leaves fp32's range
    if (temperature != 0.f && !(temperature >= 1e-30f && temperature <= 1e30f))
        return fail(TFM_EINVAL, "temperature must be 0 or in [1e-30, 1e30]");
    const bool greedy = temperature == 0.f;
    if (ld_target < V || ld_target % 4) return fail(TFM_EINVAL, "ld_target must be >= V and a multiple of 4");
    if (!greedy && ((K && (ld_draft < V || ld_draft % 4)) || ld_noise < V || ld_noise % 4))
        return fail(TFM_EINVAL, "ld_draft and ld_noise must be >= V and multiples of 4");
    if (B == 0) return TFM_OK;
    if (!target || !tokens || !n_accepted || !workspace || (K && !draft) ||
        (!greedy && (!noise || (K && (!draft_logits || !u)))))
        return fail(TFM_EINVAL, "NULL pointer");
    if (!aligned(target, 16) || !aligned(workspace, 16) ||
        (!greedy && (!aligned(noise, 16) || (K && !aligned(draft_logits, 16)))))
        return fail(TFM_EINVAL, "logits, noise and workspace must be 16-byte aligned");
    if (!aligned(draft, 4) || !aligned(n_draft, 4) || !aligned(u, 4) || !aligned(tokens, 4) || !aligned(n_accepted, 4))
        return fail(TFM_EINVAL, "draft, n_draft, u, tokens and n_accepted must be 4-byte aligned");
    if (workspace_bytes < tfm::verify_workspace_bytes(B, K, V)) return fail(TFM_EINVAL, "workspace too small");
    if (!tfm::device_error_word()) return fail(TFM_ECUDA, "device error word unavailable");
    tfm::VerifyArgs a{};
    a.target = target;
    a.ld_target = ld_target;
    a.dlogits = draft_logits;
    a.ld_draft = ld_draft;
    a.draft = draft;
    a.n_draft = n_draft;
    a.u = u;
    a.noise = noise;
    a.ld_noise = ld_noise;
    a.B = B;
    a.K = K;
    a.V = V;
    a.temperature = temperature;
    a.tokens = tokens;
    a.n_accepted = n_accepted;
    a.ws = workspace;
    const cudaError_t e = tfm::launch_verify_draft(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TFM_OK : cuda_fail(e, "verification launch");
}

}  // extern "C"
