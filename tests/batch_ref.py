"""Plain 64-bit forms of the batched-serving operators, for the tests."""
import numpy as np
import torch


def softmax_rows(s):
    """Softmax of the last axis in float64; a row without any finite score gives zeros."""
    m = s.max(axis=-1, keepdims=True, initial=-np.inf)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isneginf(s), 0.0, np.exp(s - np.where(np.isneginf(m), 0.0, m)))
    t = e.sum(-1, keepdims=True)
    return np.divide(e, t, out=np.zeros_like(e), where=t > 0)


def f64(t):
    return t.detach().double().cpu().numpy()


def packed(q, k, v, lens, window=0, scale=None):
    """[rows, H, dh] of the sequences' rows, one behind the other; keys a row does not see are not touched."""
    q, k, v = f64(q), f64(k), f64(v)
    H, dh = q.shape[1:]
    G = H // k.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    out, a = np.zeros((sum(lens), H, dh)), 0
    for L in lens:
        i, j = np.arange(L)[:, None], np.arange(L)[None, :]
        seen = (j <= i) & ((j > i - window) if window else True)
        for h in range(H):
            with np.errstate(invalid="ignore"):
                s = q[a:a + L, h] @ k[a:a + L, h // G].T * scale
            p = softmax_rows(np.where(seen, s, -np.inf))
            out[a:a + L, h] = weighted(p, v[a:a + L, h // G], seen)
        a += L
    return out


def weighted(p, v, seen):
    """p @ v where a value that is not seen does not count, whatever it is."""
    if np.isfinite(v).all():
        return p @ v
    out = np.zeros((p.shape[0], v.shape[1]))
    for i in range(p.shape[0]):
        out[i] = p[i, seen[i]] @ v[seen[i]]
    return out


def prefix(q, kp, vp, kc, vc, lens, prefix_len, scale=None):
    """[B, T, H*dh]."""
    q, kp, vp, kc, vc = (f64(x) for x in (q, kp, vp, kc, vc))
    B, H, T, dh = q.shape
    G = H // kc.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    out = np.zeros((B, T, H, dh))
    for b in range(B):
        for h in range(H):
            for t in range(T):
                n = max(0, lens[b] - (T - 1 - t))
                k = np.concatenate([kp[h // G, :prefix_len], kc[b, h // G, :n]])
                v = np.concatenate([vp[h // G, :prefix_len], vc[b, h // G, :n]])
                if len(k):
                    out[b, t, h] = softmax_rows((k @ q[b, h, t] * scale)[None])[0] @ v
    return out.reshape(B, T, H * dh)


def verify(target, dlogits, draft, n_draft, u, noise, V, temperature):
    """(tokens [B, K+1], n_accepted [B]) by loops; NaN logits have no weight, +inf takes all of it."""
    target, noise = f64(target)[:, :V], None if noise is None else f64(noise)[:, :V]
    dlogits = None if dlogits is None else f64(dlogits)[:, :V]
    u = None if u is None else f64(u)
    draft = draft.cpu().numpy()
    B, K = draft.shape

    def probs(z):
        z = np.where(np.isnan(z), -np.inf, z)
        m = z.max()
        if m == -np.inf:
            return np.zeros(V)
        w = (z == np.inf).astype(float) if m == np.inf else np.exp((z - m) / temperature)
        return w / w.sum()

    def race(w, b):
        ok = (noise[b] > 0) & (w > 0)
        if not ok.any():
            return -1
        s = np.where(ok, w / np.where(noise[b] > 0, noise[b], 1.0), -1.0)
        return int(np.argmax(s))

    tokens, count = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = 0
        while True:
            z = target[b * (K + 1) + n]
            last = n == n_draft[b]
            x = -1 if last else int(draft[b, n])
            if temperature == 0:
                z = np.where(np.isnan(z), -np.inf, z)
                new = int(np.argmax(z)) if z.max() > -np.inf else -1
                if last or x != new or new < 0:
                    break
            else:
                p = probs(z)
                if last:
                    new = race(p, b)
                    break
                q = probs(dlogits[b * K + n])
                if not (0 <= x < V and u[b, n] * q[x] < p[x]):
                    new = race(np.maximum(p - q, 0), b)
                    if new < 0:
                        new = race(p, b)
                    break
            tokens[b, n] = x
            n += 1
        tokens[b, n] = new
        count[b] = n
    return tokens, count


def bound(v, dh, keys, smax, dtype):
    """How far an output may be off, from the roundings alone.  o is an average of
    values: an error e relative to each weight moves it by at most e max|v|.  A score
    of dh products has an error of dh 2^-24 of the sum of their magnitudes (at most
    smax, scaled), which the weight takes over, its sum too; a sum over the keys adds
    keys 2^-24 twice (weights, products), exponential, scale and division a few more.
    In bf16 the weights are rounded (2^-8) and so is the output (2^-8)."""
    e = (2 * dh * smax + 2 * keys + 64) * 2.0 ** -24
    if dtype == torch.bfloat16:
        e = (1 + e) * (1 + 2.0 ** -8) ** 2 - 1
    return e * float(np.abs(v[np.isfinite(v)]).max(initial=0.0))
