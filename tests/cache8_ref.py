"""Plain 64-bit forms of the 8-bit cache's operators, for the tests."""
import numpy as np
import torch

from batch_ref import f64, softmax_rows

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}

# every e4m3 value that is not negative, by its code
_E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])


def rope(x, positions, inv, interleaved, mscale):
    """x [T, heads, dh] turned, in float64; and the sum of the magnitudes that each value is made of."""
    y, size = f64(x).copy(), np.abs(f64(x))
    r = len(inv)
    a, b = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
    # the angle modulo one turn, the product in extended precision
    turn = np.longdouble(2) * np.arctan2(np.longdouble(0), np.longdouble(-1))
    ang = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv, np.longdouble)[None]
    ang = (ang - turn * np.floor(ang / turn)).astype(np.float64)[:, None]
    c, s, p, q = np.cos(ang) * mscale, np.sin(ang) * mscale, y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = p * c - q * s, p * s + q * c
    size[..., a] = size[..., b] = (np.abs(p) + np.abs(q)) * abs(mscale)
    return y, size


def code(y, dtype):
    """The codes' values nearest to quotients y (float64), ties to the even code; NaN is 0."""
    y = np.where(np.isnan(y), 0.0, y)
    if dtype == torch.int8:
        return np.clip(np.rint(y), -127, 127)
    a = np.minimum(np.abs(y), 448.0)
    mid = (_E4M3[1:] + _E4M3[:-1]) / 2
    i = np.searchsorted(mid, a)
    i = i + ((i < len(mid)) & (a == mid[np.minimum(i, len(mid) - 1)]) & (i % 2 == 1))
    return np.copysign(_E4M3[i], y)


def write(x, codes, scales, lens, new, block, dtype):
    """codes (values, float64 [B, Hkv, max_seq, dh]) and scales [B, Hkv, nblk] after the rows x [T, Hkv, dh] have joined."""
    x, codes, scales, top, a = f64(x), codes.copy(), scales.astype(np.float64).copy(), TOP[dtype], 0
    for b, (L, n) in enumerate(zip(lens, new)):
        rows = x[a:a + n]
        a += n
        if not 0 <= n <= L <= codes.shape[2]:
            continue
        start = L - n
        for j in range(start // block, -(-L // block) if n else 0):
            lo, hi = max(j * block, start), min((j + 1) * block, L)
            part = rows[lo - start:hi - start]                           # [rows, Hkv, dh]
            for h in range(codes.shape[1]):
                y = part[:, h]
                m = np.abs(y[np.isfinite(y)]).max(initial=0.0)
                need = max(float(np.float32(m / top)), 2.0 ** -126) if m > 0 else 0.0
                old = scales[b, h, j]
                if lo > j * block and old > 0:
                    s = old
                    while s < need:
                        s *= 2
                    if s > old:
                        codes[b, h, j * block:lo] = code(codes[b, h, j * block:lo] * (old / s), dtype)
                else:
                    s = need
                scales[b, h, j] = s
                with np.errstate(invalid="ignore"):
                    codes[b, h, lo:hi] = code(y / s, dtype) if s > 0 else 0.0
    return codes, scales


def values(codes, scales, block):
    """float64 [B, Hkv, max_seq, dh] of tensors or arrays."""
    c = f64(codes.float()) if isinstance(codes, torch.Tensor) else codes
    s = f64(scales) if isinstance(scales, torch.Tensor) else scales
    return c * np.repeat(s, block, 2)[:, :, :c.shape[2], None]


def attention(q, k, v, lens, new, window=0, scale=None):
    """[T, H, dh]: rows q over the caches' values k, v [B, Hkv, max_seq, dh]; what a row does not see is not touched."""
    q = f64(q)
    out, a = np.zeros(q.shape), 0
    H, dh = q.shape[1:]
    G = H // k.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    for b, (L, n) in enumerate(zip(lens, new)):
        for t in range(n):
            p = L - n + t
            lo = max(0, p - window + 1) if window else 0
            for g in range(k.shape[1] if p >= 0 else 0):
                s = q[a + t, g * G:(g + 1) * G] @ k[b, g, lo:p + 1].T * scale
                out[a + t, g * G:(g + 1) * G] = softmax_rows(s) @ v[b, g, lo:p + 1]
        a += n
    return out


def bound(k, v, q, lens, scale=None):
    """How far an output may be off, from the roundings alone.  A score of dh exact products is summed in fp32 (2 dh
    2^-24 of the sum of their magnitudes, at most smax, should each addition truncate), q's small elements are off by
    2^-24 of its largest (sqrt(dh) 2^-24 smax), scaling adds four roundings: below 3 dh 2^-24 smax, relative to the weight,
    once in the products and once in the sum.  The sums over the keys add keys 2^-24 each, the scales two roundings,
    exponentials, joins and the division some more.  Weights are rounded to fp16 (2^-11), the output to bf16 (2^-8)."""
    dh = q.shape[-1]
    keys = max(list(lens) + [1])
    norm = lambda x: float(np.sqrt((x ** 2).sum(-1).max(initial=0.0)))
    seen = [(k[b, :, :max(L, 0)], v[b, :, :max(L, 0)]) for b, L in enumerate(lens)]
    smax = norm(f64(q)) * max(norm(x) for x, _ in seen) * (dh ** -0.5 if scale is None else scale)
    e = (6 * dh * smax + 2 * keys + 64) * 2.0 ** -24
    e = (1 + e) * (1 + 2.0 ** -11) * (1 + 2.0 ** -8) - 1
    return e * max(float(np.abs(y).max(initial=0.0)) for _, y in seen)
