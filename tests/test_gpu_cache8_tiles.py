"""Attention over the 8-bit cache: that every tile of 64 positions is counted once, wherever the runs that the jobs are cut
into begin and end."""
import numpy as np
import pytest

from batch_ref import f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402
from test_gpu_cache8_attention import _cache, _call, _q, _with_room  # noqa: E402

BF, I8, E4 = torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


def _case(codes, lens, H, Hkv, T, dh, block, window):
    """Cache, queries, outputs in 64 bits, their tolerance.  Coordinate c of kv head h has the code 64 in the tiles number h dh + c
    modulo Hkv dh and zero in all others; scores are one number for a tile (up to 1 in magnitude, by the first coordinate).
    So a tile that is left out, or counted twice, moves the coordinate of its own by a good part of its value: what the
    assertion at the end holds each tile to."""
    B, n = len(lens), max(max(lens), 1)
    rng = np.random.default_rng(n + dh)
    tiles, channels = -(-n // 64), Hkv * dh
    tile = np.arange(n) // 64
    at = tile % channels
    level = rng.integers(-8, 9, (B, tiles))                     # scores of a tile, in eighths
    vs = ((1 + rng.random((B, Hkv, -(-n // block)))) / 64).astype(np.float32)
    kc = torch.zeros(B, Hkv, n, dh, dtype=torch.int8, device="cuda")
    vc = torch.zeros_like(kc)
    byte = torch.from_numpy(level[:, tile]).float().cuda().to(codes).view(torch.int8)
    kc[:, :, :, 0] = byte[:, None]
    vc[:, torch.from_numpy(at // dh).cuda(), torch.arange(n, device="cuda"), torch.from_numpy(at % dh).cuda()] = \
        64 if codes == I8 else 0x68                             # 64 in e4m3
    cache = [kc.view(codes), vc.view(codes), torch.full((B, Hkv, -(-n // block)), 0.125, device="cuda"), torch.from_numpy(vs).cuda()]
    strength = np.array([1.0, 0.0, -1.0, 0.5])                  # of a query head
    q = torch.zeros(B * T, H, dh, dtype=BF, device="cuda")
    q[:, :, 0] = torch.from_numpy(strength[np.arange(H) % 4]).to(BF).cuda()
    G = H // Hkv
    want, tol = np.zeros((B * T, H, dh)), np.zeros((B * T, H, dh))
    # 2^-8: the output's rounding to bf16.  2^-10: the weights' to fp16, in the products and in their sum.  The sums over the
    # tiles: two additions each, some more where parts are joined; scores of 1 and their exponentials: below 2^-20.
    rel = 2.0 ** -8 + 2.0 ** -10 + (2 * tiles + 400) * 2.0 ** -24
    for b, L in enumerate(lens):
        for t in range(T):
            p = L - T + t
            pos = np.arange(max(0, p - window + 1) if window else 0, p + 1)
            if len(pos) == 0:
                continue
            for s in range(min(4, H)):
                w = np.exp(level[b, tile[pos]] / 8 * strength[s])
                for h in range(s, H, 4):
                    v = vs[b, h // G, pos // block].astype(np.float64)
                    part = np.bincount(tile[pos], w * v * 64, tiles) / w.sum()
                    each = np.zeros(channels)
                    np.add.at(each, np.arange(tiles) % channels, part)
                    r = b * T + t
                    want[r, h] = each[h // G * dh:(h // G + 1) * dh]
                    # int8 codes are multiplied as c + 128, and the bias is taken off: 17 terms, at most 383 steps together, each
                    # addition truncated at 2^-23 of them
                    tol[r, h] = rel * want[r, h] + (17 * 383 * 2.0 ** -23 * (w * v).sum() / w.sum() if codes == I8 else 0.0)
                    mine = (np.arange(tiles) % channels) // dh == h // G
                    share = part[mine & (part > 0)]
                    whole = tol[r, h][np.arange(tiles)[mine & (part > 0)] % channels % dh]
                    counts = np.bincount(tile[pos], minlength=tiles)[mine & (part > 0)] == 64
                    assert (share[counts] > 2 * whole[counts]).all()
    return cache, q, want, tol


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("lens,H,Hkv,T,dh,block,window,room", [
    ([70001, 3, 64, 65], 8, 1, 1, 128, 128, 0, 0), ([70001, 3], 2, 2, 1, 64, 64, 0, 0), ([30000, 29999], 8, 4, 9, 64, 32, 0, 0),
    ([1000, 130], 8, 2, 1, 128, 32, 0, 0), ([20011], 32, 1, 1, 128, 64, 0, 100032), ([20011], 16, 1, 1, 64, 16, 0, 300032),
    ([20011, 7], 24, 1, 1, 32, 128, 0, 250112), ([20011], 8, 1, 3, 128, 64, 0, 120064), ([20011], 16, 1, 8, 128, 64, 0, 0),
    ([0, 1, 63, 64, 65, 127, 128, 129, 500, 5000, 2100, 777, 4096, 4095, 4097, 3, 0, 2000], 4, 4, 1, 64, 64, 0, 0),
    ([5000, 1200, 60, 3000, 4999] * 6, 8, 4, 2, 32, 16, 1000, 0), ([700, 70, 800, 64] * 40, 8, 8, 1, 64, 16, 0, 0),
    ([500, 70, 300, 64], 12, 12, 1, 64, 16, 0, 0), ([20011], 1, 1, 1, 128, 128, 15000, 0)], ids=lambda x: str(x)[:40])
def test_every_tile_counts_once(lens, H, Hkv, T, dh, block, window, room, codes):
    """Whole and cut jobs, jobs of 8 to 32 rows and several of them for a sequence, sequences side by side, windows."""
    cache, q, want, tol = _case(codes, lens, H, Hkv, T, dh, block, window)
    if room:
        n = -(-max(lens) // block) * block
        pad = n - cache[0].shape[2]
        cache = [torch.nn.functional.pad(c.view(torch.int8), (0, 0, 0, pad)).view(codes) for c in cache[:2]] + cache[2:]
        cache = _with_room(cache, block, room // block * block)
    o = f64(_call(q, cache, lens, block, window=window, scale=1.0))
    off = np.abs(o - want) - tol
    assert (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:5])


def _rows_and_tolerances(q, cache, lens, T, block, window):
    """Outputs in 64 bits and what the roundings can make of each of them: with o = sum w v, weights off by a part d and scores by
    e move it by at most sum w (d + e) |v - o|.  d: 2^-11, the weights' rounding to fp16, or below 2^-21 of the row's largest weight
    2^-32 of that.  e: the scores' sums of dh products, each addition truncated at 2^-23 of all of their magnitudes (int8 codes are
    taken as c + 128, and the bias is one term more), and six roundings of the score itself.  The products with the values: 17
    terms in the same way, for int8 up to 383 steps.  The sums over the tiles: two additions of fp32 each, some more where parts are
    joined.  The output is rounded to bf16, 2^-8."""
    B, Hkv = len(lens), cache[0].shape[1]
    H, dh = q.shape[1:]
    G, int8 = H // Hkv, cache[0].dtype == I8
    kc, vc, ks, vs = (f64(c.float()) for c in cache)
    qq = f64(q)
    want, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b, L in enumerate(lens):
        for t in range(T):
            p = L - T + t
            j = np.arange(max(0, p - window + 1) if window else 0, p + 1)
            for h in range(H if len(j) else 0):
                g, r = h // G, b * T + t
                sk, sv = ks[b, g, j // block], vs[b, g, j // block]
                k, v = kc[b, g, j], vc[b, g, j] * sv[:, None]
                f = dh ** -0.5 * sk
                s = k @ qq[r, h] * f
                e = ((np.abs(k) + (256 if int8 else 0)) @ np.abs(qq[r, h]) * f * (dh + 1) + 6 * np.abs(s) + 8) * 2.0 ** -23
                w = np.exp(s - s.max())
                least = w.max() * 2.0 ** -32 / w.sum()
                w /= w.sum()
                o = w @ v
                off = np.abs(v - o)
                tol[r, h] = ((w * (2.0 ** -11 + e)) @ off + least * off.sum(0)) * (1 + 2.0 ** -9)
                tol[r, h] += 17 * 2.0 ** -23 * ((w * sv * 383).sum() if int8 else w @ np.abs(v))
                tol[r, h] += (2 * (len(j) // 64) + 400) * 2.0 ** -24 * (w @ np.abs(v))
                tol[r, h] = tol[r, h] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o)
                want[r, h] = o
    return want, tol


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("lens,H,Hkv,T,dh,block,window", [
    ([1000, 130], 8, 2, 1, 128, 32, 0), ([3000, 64, 2999], 4, 4, 1, 64, 16, 0), ([3000, 5], 8, 1, 4, 64, 128, 0),
    ([2500], 16, 1, 2, 32, 64, 0), ([1500, 1501, 90], 8, 2, 3, 128, 16, 700), ([20000], 2, 2, 1, 128, 64, 0),
    ([700, 33, 1, 500, 64, 128] * 5, 8, 4, 1, 64, 64, 0)], ids=lambda x: str(x)[:30])
def test_rows_within_their_own_tolerance(lens, H, Hkv, T, dh, block, window, codes):
    """Each output within what its own row's weights and values allow, a few thousandths of itself."""
    cache = _cache(61, len(lens), Hkv, max(lens) + 3, dh, block, codes)
    q = _q(61, len(lens) * T, H, dh)
    want, tol = _rows_and_tolerances(q, cache, lens, T, block, window)
    off = np.abs(f64(_call(q, cache, lens, block, window=window)) - want)
    assert (off <= tol).all(), (off - tol).max()
