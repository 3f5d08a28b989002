"""Attention over the 8-bit cache on the GPU (tfm_cache8_attention) against its plain form in
64 bits, and a serving program's steps with rotary positions, write and attention."""
import numpy as np
import pytest

from batch_ref import f64
from cache8_ref import TOP, attention, bound, rope, values, write

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402

BF, I8, E4 = torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


def _ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _ends(new):
    return _ints(np.cumsum([0] + list(new)))


def _bytes(n):
    return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")


def _cache(seed, B, Hkv, room, dh, block, dtype):
    g = torch.Generator().manual_seed(seed)
    top = TOP[dtype]
    out, scales = [], []
    for _ in "kv":
        c = (torch.randn(B, Hkv, room, dh, generator=g) * top / 3).clamp(-top, top)
        out.append((c.round() if dtype == I8 else c).to(dtype).cuda())
        scales.append((torch.exp2(torch.randn(B, Hkv, -(-room // block), generator=g)) * 3 / top).cuda())
    return [*out, *scales]


def _q(seed, T, H, dh):
    return torch.randn(T, H, dh, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def _call(q, cache, lens, block, new=None, max_new=None, window=0, scale=0.0):
    B, Hkv = len(lens), cache[0].shape[1]
    cu = None if new is None else _ends(new)
    most = max_new or (max(max(new), 1) if new is not None else max(q.shape[0] // B, 1))
    ws = _bytes(tfm.cache8_attention_workspace_bytes(B, q.shape[1], Hkv, most, q.shape[2]))
    o = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    tfm.cache8_attention(q, *cache, o, _ints(lens), ws, block, cu_seqlens=cu, max_new=most, window=window, scale=scale)
    torch.cuda.synchronize()
    return o


def _check(o, q, cache, lens, block, new, window=0, scale=None):
    k, v = values(cache[0], cache[2], block), values(cache[1], cache[3], block)
    want = attention(q, k, v, lens, new, window, scale)
    got = f64(o)
    assert np.isfinite(got).all()
    worst, limit = np.abs(got - want).max(initial=0.0), bound(k, v, q, lens, scale)
    assert worst <= limit, (worst, limit)


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dh,block", [(32, 16), (64, 64), (128, 32), (128, 128), (64, 16)])
@pytest.mark.parametrize("H,Hkv,T", [(4, 4, 1), (8, 2, 1), (8, 1, 1), (6, 2, 5), (4, 4, 3), (16, 1, 8), (3, 3, 128), (16, 1, 2), (20, 2, 4)])
@pytest.mark.parametrize("lens", [[1], [1, 64, 65, 0, 200, 16, 17], [15, 31, 33, 128, 129, 127], [1000, 130], [0, 0]], ids=str)
def test_sizes(lens, H, Hkv, T, dh, block, codes):
    cache = _cache(dh + T, len(lens), Hkv, max(lens) + 3, dh, block, codes)
    q = _q(T, len(lens) * T, H, dh)
    _check(_call(q, cache, lens, block), q, cache, lens, block, [T] * len(lens))


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("window", [1, 5, 16, 63, 64, 100, 5000])
def test_windows(window, dh, codes):
    lens = [1, 64, 300, 129, 0, 77, 1000]
    for H, Hkv, T in ((8, 2, 1), (4, 4, 4), (16, 1, 8)):
        cache = _cache(window, len(lens), Hkv, 1003, dh, 32, codes)
        q = _q(window, len(lens) * T, H, dh)
        _check(_call(q, cache, lens, 32, window=window), q, cache, lens, 32, [T] * len(lens), window)


@pytest.mark.parametrize("codes", [I8, E4])
def test_ragged_rows(codes):
    """Sequences with none to max_new new rows, and rows behind the last sequence, which stay as they were."""
    lens, new = [100, 7, 0, 300, 64, 3], [5, 0, 0, 1, 8, 3]
    for H, Hkv, dh in ((8, 2, 128), (12, 12, 64), (16, 1, 32)):
        cache = _cache(1, 6, Hkv, 301, dh, 16, codes)
        q = _q(2, sum(new) + 4, H, dh)
        for max_new in (8, 8 if H == 16 else 20):
            o = _call(q, cache, lens, 16, new, max_new)
            _check(o[:sum(new)], q[:sum(new)], cache, lens, 16, new)
            assert (o[sum(new):] == 7.0).all()


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("T", [1, 4])
def test_what_is_not_seen_is_not_looked_at(T, codes):
    lens, block = [4, 70, 0, 64, 130], 32
    for window in (0, 20):
        cache = _cache(T, 5, 2, 200, 128, block, codes)
        q = _q(T, 5 * T, 8, 128)
        clean = _call(q, cache, lens, block, window=window)
        for c in (0x7f, 0xff, 0x80):
            for s in (float("nan"), float("inf")):
                other = [t.clone() for t in cache]
                for b, n in enumerate(lens):
                    lo = max(0, n - T - window + 1) if window else 0
                    for t in other[:2]:
                        t.view(torch.uint8)[b, :, n:] = c
                        t.view(torch.uint8)[b, :, :lo] = c
                    for t in other[2:]:
                        t[b, :, -(-n // block):] = s
                        t[b, :, :lo // block] = s
                assert torch.equal(_call(q, other, lens, block, window=window), clean)


def test_new_rows_do_not_see_those_behind_them():
    cache = _cache(7, 3, 2, 100, 64, 16, I8)
    lens, q = [100, 5, 64], _q(7, 12, 4, 64)
    clean = _call(q, cache, lens, 16).view(3, 4, 4, 64)
    for back in (1, 2, 3):
        other = [t.clone() for t in cache]
        for b, n in enumerate(lens):
            other[0][b, 0, n - back] = -other[0][b, 0, n - back]
            other[1][b, 1, n - back] = 127
        o = _call(q, other, lens, 16).view(3, 4, 4, 64)
        assert torch.equal(o[:, :4 - back], clean[:, :4 - back])
        assert not torch.equal(o[:, 4 - back:], clean[:, 4 - back:])


def test_one_row_does_not_reach_another():
    """NaN and infinities in one row of q stay there, whether rows share a tile or not."""
    for H, Hkv, T in ((8, 2, 1), (8, 1, 4)):
        lens = [100, 40, 257]
        cache = _cache(9, 3, Hkv, 300, 64, 64, E4)
        q = _q(9, 3 * T, H, 64)
        clean = _call(q, cache, lens, 64)
        for bad in (float("nan"), float("inf")):
            x = q.clone()
            x[T, 1, 3] = bad
            o = _call(x, cache, lens, 64)
            same = torch.ones_like(o, dtype=torch.bool)
            same[T, 1] = False
            assert torch.equal(o[same], clean[same]) and not torch.isfinite(o[T, 1]).any()


@pytest.mark.parametrize("codes", [I8, E4])
def test_large_and_small_scores(codes):
    """Scores of hundreds (one key takes all), rows of q with elements 2^20 apart, tiny rows, rows of zeros."""
    lens, block = [200, 333], 16
    cache = _cache(11, 2, 2, 340, 128, block, codes)
    for factor in (40.0, 2.0 ** -120, 2.0 ** 20, 0.0):
        q = (_q(11, 2, 8, 128).float() * factor).to(BF)
        s = dict(scale=2.0 ** -22) if factor == 2.0 ** 20 else {}
        _check(_call(q, cache, lens, block, **s), q, cache, lens, block, [1, 1], 0, s.get("scale"))
    q = (_q(12, 2, 8, 128).float() * torch.exp2(torch.arange(128, device="cuda") % 21 - 20.0)).to(BF)
    _check(_call(q, cache, lens, block, scale=2.0), q, cache, lens, block, [1, 1], 0, 2.0)
    # a far larger key late in the sequence, and values whose blocks differ by 2^30
    cache[2][:, :, 15:] *= 50.0
    cache[3][:, :, 3] *= 2.0 ** 30
    cache[3][:, :, 4] *= 2.0 ** -30
    q = _q(13, 2, 8, 128)
    _check(_call(q, cache, lens, block), q, cache, lens, block, [1, 1])


def test_agrees_with_the_16_bit_cache():
    """Codes and scales that are powers of two are bf16 numbers: the same attention over them by tfm_prefix_attention, each
    side within its roundings (that one rounds weights and output to bf16)."""
    lens = [333, 12, 130]
    cache = _cache(15, 3, 4, 340, 64, 64, I8)
    for s in cache[2:]:
        s.copy_(torch.exp2(torch.log2(s).round()))
    q = _q(15, 3, 8, 64)
    o = _call(q, cache, lens, 64)
    k, v = (torch.from_numpy(values(c, s, 64)).to(BF).cuda() for c, s in ((cache[0], cache[2]), (cache[1], cache[3])))
    none = torch.empty(4, 0, 64, dtype=BF, device="cuda")
    ws = _bytes(tfm.prefix_attention_workspace_bytes(3, 8, 4, 1, 64))
    p = torch.empty(3, 1, 512, dtype=BF, device="cuda")
    tfm.prefix_attention(q.view(3, 8, 1, 64), none, none, k, v, p, _ints(lens), ws)
    torch.cuda.synchronize()
    assert float((o.view(3, 512).float() - p.view(3, 512).float()).abs().max()) <= 3.3 * 2.0 ** -8 * float(v.abs().max())


def test_lengths_and_offsets_out_of_range():
    cache = _cache(2, 3, 2, 40, 64, 16, I8)
    q = _q(2, 3, 4, 64)
    o = _call(q, cache, [41, -1, 40], 16)
    with pytest.raises(tfm.TfmError) as e:
        tfm.device_status()
    assert e.value.status == tfm.TFM_EINVAL
    _check(o, q, cache, [0, 0, 40], 16, [1, 1, 1])
    q = _q(3, 12, 4, 64)
    whole = torch.full((36, 4, 64), 7.0, dtype=BF, device="cuda")
    ws = _bytes(3 * 4096 + tfm.cache8_attention_workspace_bytes(3, 4, 2, 5, 64))
    for cu in ([0, 6, 8, 12], [0, 5, 3, 8], [0, 4, 8, 13], [-2, 3, 5, 9], [0, 2 ** 31 - 1, -2 ** 31, 12], [12, 8, 4, 0]):
        whole.fill_(7.0)
        tfm.cache8_attention(q, *cache, whole[12:24], _ints([40, 30, 20]), ws[4096:-8192], 16, cu_seqlens=_ints(cu), max_new=5)
        with pytest.raises(tfm.TfmError) as e:
            tfm.device_status()
        assert e.value.status == tfm.TFM_EINVAL
        assert (whole[:12] == 7.0).all() and (whole[24:] == 7.0).all()
        assert (ws[:4096] == 0xff).all() and (ws[-8192:] == 0xff).all()
        for b in range(3):
            if not 0 <= cu[b] <= cu[b + 1] <= 12 or cu[b + 1] - cu[b] > 5:
                continue
            n = cu[b + 1] - cu[b]
            one = [t[b:b + 1] for t in cache]
            rows = slice(cu[b], cu[b + 1])
            if cu == [0, 6, 8, 12]:
                _check(whole[12:24][rows], q[rows], one, [[40, 30, 20][b]], 16, [n])


def test_strides_of_a_fused_projection():
    lens, T = [70, 33, 128], 3
    cache = _cache(4, 3, 2, 130, 128, 64, E4)
    x = torch.randn(9, 12, 128, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    q = x[:, :8]
    heads = torch.full((8, 9, 128), 7.0, dtype=BF, device="cuda")
    ws = _bytes(tfm.cache8_attention_workspace_bytes(3, 8, 2, 3, 128))
    tfm.cache8_attention(q, *cache, heads.transpose(0, 1), _ints(lens), ws, 64)
    torch.cuda.synchronize()
    assert torch.equal(heads.transpose(0, 1), _call(q.contiguous(), cache, lens, 64))
    _check(heads.transpose(0, 1), q, cache, lens, 64, [T] * 3)


def test_large_batches_and_long_caches():
    lens = [(i * 37) % 90 for i in range(1500)]
    cache = _cache(12, 1500, 2, 91, 32, 16, I8)
    q = _q(12, 1500, 4, 32)
    _check(_call(q, cache, lens, 16), q, cache, lens, 16, [1] * 1500)
    for H, Hkv, T, dh in ((8, 1, 1, 128), (8, 4, 9, 64), (2, 2, 1, 64)):
        lens = [70001, 3]
        cache = _cache(13, 2, Hkv, 70010, dh, 128, E4)
        q = _q(13, 2 * T, H, dh)
        o = _call(q, cache, lens, 128)
        _check(o, q, cache, lens, 128, [T] * 2)
        for _ in range(3):
            assert torch.equal(_call(q, cache, lens, 128), o)


def test_offsets_beyond_32_bits():
    """Sequences at the end of a cache of more than 2^32 codes."""
    room, lens = 4_400_001, [100, 4_400_001]
    kc, vc = (torch.zeros(2, 4, room, 128, dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(2, 4, -(-room // 128), device="cuda") for _ in "kv")
    small = _cache(16, 2, 4, 257, 128, 128, I8)
    at = room // 128 * 128 - 128                              # whole blocks, the last one of a single position
    n = room - at
    for big, c in ((kc, small[0]), (vc, small[1])):
        big[1, :, at:] = c[1, :, :n]
        big[0, :, :100] = c[0, :, :100]
    for big, s in ((ks, small[2]), (vs, small[3])):
        big[1, :, at // 128:] = s[1, :, :big.shape[2] - at // 128]
        big[0, :, 0] = s[0, :, 0]
    q = _q(16, 2, 8, 128)
    o = _call(q, [kc, vc, ks, vs], lens, 128, window=n)
    _check(o, q, small, [100, n], 128, [1, 1])


def test_graphs_share_a_workspace_and_follow_the_lengths():
    cache = _cache(17, 4, 2, 400, 128, 32, I8)
    q = _q(17, 8, 8, 128)
    lens, ws = _ints([5, 100, 400, 77]), _bytes(tfm.cache8_attention_workspace_bytes(4, 8, 2, 2, 128))
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
    graphs, s = [], torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for o, w in ((o1, 0), (o2, 50)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                tfm.cache8_attention(q, *cache, o, lens, ws, 32, window=w)
            graphs.append(g)
        for new in ([5, 100, 400, 77], [400] * 4, [0, 2, 0, 399], [0] * 4):
            lens.copy_(_ints(new))
            o1.fill_(7.0), o2.fill_(7.0)
            for g in graphs + graphs[::-1]:
                g.replay()
            s.synchronize()
            assert torch.equal(o1, _call(q, cache, new, 32)) and torch.equal(o2, _call(q, cache, new, 32, window=50))
            _check(o1, q, cache, new, 32, [2] * 4)


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("H,Hkv,dh,T", [(8, 4, 32, 1), (16, 4, 128, 2), (12, 12, 64, 1)])
def test_calls_behind_one_another_as_calls_apart(H, Hkv, dh, T, codes):
    """Rotation in place, write, attention and reading back, launched behind one another and recorded, many layers of
    them: the bits of the same calls with the device waited for in between."""
    B, room, block, layers = 48, 150, 16, 6
    g = torch.Generator().manual_seed(dh)
    inv = tfm.rope_frequencies(10000.0, dh)[0].cuda()
    lens = torch.randint(T, room, (B,), generator=g, dtype=torch.int32).cuda()
    positions = (lens[:, None] - T + torch.arange(T, device="cuda", dtype=torch.int32)).flatten().contiguous()
    rows = torch.randn(layers, B * T, H + 2 * Hkv, dh, generator=g).to(BF).cuda()
    caches = [_cache(i, B, Hkv, room, dh, block, codes) for i in range(layers)]
    ws = _bytes(tfm.cache8_attention_workspace_bytes(B, H, Hkv, T, dh))

    def layer(x, cache, o, back, wait):
        q, k, v = x.split((H, Hkv, Hkv), 1)
        for call in (lambda: tfm.rope_rows(q, k, q, k, positions, inv),
                     lambda: tfm.cache8_write(k, v, *cache, lens, block),
                     lambda: tfm.cache8_attention(q, *cache, o, lens, ws, block),
                     lambda: tfm.cache8_read(*cache, *back, lens, block)):
            call()
            if wait:
                torch.cuda.synchronize()

    def buffers():
        return (rows.clone(), [[t.clone() for t in c] for c in caches],
                torch.zeros(layers, B * T, H, dh, dtype=BF, device="cuda"),
                torch.zeros(layers, 2, B * T, Hkv, dh, dtype=BF, device="cuda"))

    x, cs, want, back = buffers()
    for i in range(layers):
        layer(x[i], cs[i], want[i], back[i], True)
    for recorded in (False, True, True):
        y, ds, o, b = buffers()
        if recorded:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
                for i in range(layers):
                    layer(y[i], ds[i], o[i], b[i], False)
            graph.replay()
        else:
            for i in range(layers):
                layer(y[i], ds[i], o[i], b[i], False)
        torch.cuda.synchronize()
        assert torch.equal(y, x) and torch.equal(o, want) and torch.equal(b, back)
        for c, d in zip(cs, ds):
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(c, d))


def test_tiles_that_reach_into_the_next_head():
    """Caches whose end lies inside a tile: what follows is the next head's or sequence's, NaN codes among it."""
    for room in (1, 63, 65, 70, 129):
        cache = _cache(room, 3, 2, room, 64, 16, E4)
        for t in cache[:2]:
            t.view(torch.uint8)[1] = 0x7f
        lens, q = [room, 0, room], _q(room, 3, 4, 64)
        clean = [t.clone() for t in cache]
        for t in clean[:2]:
            t.view(torch.uint8)[1] = 0
        o = _call(q, cache, lens, 16)
        assert torch.equal(o, _call(q, clean, lens, 16))
        _check(o, q, clean, lens, 16, [1, 1, 1])


def test_first_calls_recorded_into_a_graph():
    """In a fresh process the first call of each of the kernels is one that is recorded."""
    import subprocess
    import sys
    code = """
import sys, torch
sys.path[:0] = ['tests', '.']
import test_gpu_cache8_attention as t
from decoder_only_transformer_gb300 import tfm
for H, Hkv, T, dh in ((4, 4, 1, 128), (16, 1, 1, 64), (20, 1, 1, 128), (16, 2, 4, 128), (4, 4, 1, 32)):
    cache = t._cache(1, 2, Hkv, 2000, dh, 64, t.I8)
    lens, q = t._ints([1990, 70]), t._q(1, 2 * T, H, dh)
    ws, o = t._bytes(tfm.cache8_attention_workspace_bytes(2, H, Hkv, T, dh)), torch.zeros_like(q)
    k, v = t._q(2, 2 * T, Hkv, dh), t._q(3, 2 * T, Hkv, dh)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        tfm.cache8_write(k, v, *cache, lens, 64)
        tfm.cache8_attention(q, *cache, o, lens, ws, 64)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, t._call(q, cache, [1990, 70], 64)) and float(o.abs().max()) > 0
tfm.device_status()
print('recorded')
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "recorded" in r.stdout, r.stderr[-2000:]


def test_scales_far_apart_and_zero():
    """Blocks of V with scale zero, whose keys count in the sum of the weights, and scales that differ by 2^60; for K a
    scale of zero is a score of zero."""
    lens, block = [200, 333], 16
    for codes in (I8, E4):
        cache = _cache(21, 2, 2, 340, 128, block, codes)
        for b in (0, 5, 12):
            cache[3][:, :, b] = 0.0
        cache[2][:, :, 7] = 0.0
        for H, T in ((8, 1), (8, 3), (2, 1)):
            q = _q(21, 2 * T, H, 128)
            _check(_call(q, cache, lens, block), q, cache, lens, block, [T, T])
        for far in (2.0 ** 30, 2.0 ** -30, 2.0 ** 60):
            other = [t.clone() for t in cache]
            other[3][:, :, 3:9] *= far
            _check(_call(q, other, lens, block), q, other, lens, block, [1, 1])
        # alone, the small ones are as precise as any
        cache[3].mul_(2.0 ** -70)
        _check(_call(q, cache, lens, block), q, cache, lens, block, [1, 1])


def test_calls_on_two_streams_at_once():
    cache = _cache(18, 30, 4, 900, 64, 64, E4)
    lens = [(i * 211) % 900 for i in range(30)]
    q = _q(18, 30, 16, 64)
    want, dl = _call(q, cache, lens, 64), _ints(lens)
    size = tfm.cache8_attention_workspace_bytes(30, 16, 4, 1, 64)
    runs = [(torch.cuda.Stream(), _bytes(size), torch.zeros_like(q)) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ws, o in runs:
            tfm.cache8_attention(q, *cache, o, dl, ws, 64, stream=s)
    torch.cuda.synchronize()
    for _, _, o in runs:
        assert torch.equal(o, want)


def _with_room(cache, block, room):
    """The same positions in a cache of many more, which hold what is not to be looked at."""
    B, Hkv, n, dh = cache[0].shape
    assert n % block == 0 and room % block == 0
    out = []
    for c in cache[:2]:
        wide = torch.full((B, Hkv, room, dh), 0x7f, dtype=torch.uint8, device="cuda").view(c.dtype)
        wide[:, :, :n] = c
        out.append(wide)
    for x in cache[2:]:
        wide = torch.full((B, Hkv, room // block), float("nan"), device="cuda")
        wide[:, :, :n // block] = x
        out.append(wide)
    return out


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dh,block", [(32, 16), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("H,Hkv,T", [(8, 2, 3), (8, 2, 4), (8, 2, 5), (16, 2, 3), (8, 1, 4), (10, 2, 8), (8, 1, 16)])
@pytest.mark.parametrize("lens", [[17, 64, 65, 0, 200, 3], [128, 129, 127, 255, 33, 256]], ids=str)
def test_many_rows_of_large_caches(lens, H, Hkv, T, dh, block, codes):
    """Caches that could hold more than 16 tiles for each CTA: the rows of 2 to 4 groups of 8 share a tile.  Some sequences
    have fewer new rows."""
    B = len(lens)
    room = 128 * (152 * 16 * 3 // 2 // (B * Hkv * -(-H // Hkv * T // 8)) + 4)
    new = [T, 0, 1, T, T - 1, 2]
    cache = _cache(dh + T, B, Hkv, 256, dh, block, codes)
    q = _q(T, sum(new) + 1, H, dh)
    o = _call(q, _with_room(cache, block, room), lens, block, new, T)
    _check(o[:-1], q[:-1], cache, lens, block, new)
    assert (o[-1] == 7.0).all()


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("H,dh,T", [(8, 64, 8), (8, 64, 12), (16, 32, 8)])
def test_a_long_window_of_many_rows(H, dh, T, codes):
    """Groups of 8 rows that share tiles, whose windows begin inside them."""
    B, Hkv, room, window = 24, 4, 3200, 3000
    lens = [3200, 3001, 3007, 2999, 130, 0] + [1] * 18
    cache = _cache(21, B, Hkv, room, dh, 64, codes)
    q = _q(22, B * T, H, dh)
    o = _call(q, cache, lens, 64, [T] * B, T, window)
    n = 6
    _check(o[:n * T], q[:n * T], [x[:n].contiguous() for x in cache], lens[:n], 64, [T] * n, window)


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("H,Hkv,dh,window", [(8, 2, 128, 0), (4, 4, 64, 40), (16, 1, 32, 0)])
def test_a_serving_program(H, Hkv, dh, window, codes):
    """Prompts of different lengths prefilled from one fused projection, then steps of one and of several new tokens, some
    taken back, from a recorded graph: rotary positions, write and attention on one stream.  The cache has to be what 64
    bits make of the rotated rows, the outputs theirs within the roundings."""
    B, room, block = 4, 200, 16
    g = torch.Generator().manual_seed(H)
    inv, ms = tfm.rope_frequencies(10000.0, dh, "yarn", factor=4.0, original=64)
    dinv = inv.cuda()
    cache = _cache(19, B, Hkv, room, dh, block, codes)
    model = [(f64(c.float()), f64(s)) for c, s in ((cache[0], cache[2]), (cache[1], cache[3]))]
    ws = _bytes(tfm.cache8_attention_workspace_bytes(B, H, Hkv, 8, dh))

    def follow(x, positions, lens, new, o=None, q=None):
        """The same in 64 bits from the library's own rotated rows, which are checked against the rotation."""
        for name, raw, out in (("k", x[1], out_rows[1]), ("q", x[0], out_rows[0])):
            want, size = rope(raw, positions.tolist(), inv.tolist(), False, ms)
            assert (np.abs(f64(out) - want) <= size * 2.0 ** -20 + np.abs(want) * 2.0 ** -8 * 1.001).all(), name
        for i, rows in ((0, out_rows[1]), (1, x[2])):
            model[i] = write(rows, *model[i], lens, new, block, codes)
        for (c, s), dc, ds in zip(model, cache[:2], cache[2:]):
            assert np.array_equal(f64(ds), s) and np.array_equal(f64(dc.float()), c)
        if o is not None:
            _check(o, out_rows[0], cache, lens, block, new, window)

    # prompts: no attention over the cache here (a prompt's own attention runs packed, over the rows themselves)
    new = [30, 0, 100, 7]
    lens = list(new)
    x = torch.randn(sum(new), H + 2 * Hkv, dh, generator=g).to(BF).cuda().split((H, Hkv, Hkv), 1)
    positions = _ints(np.concatenate([np.arange(n) for n in new]))
    out_rows = [torch.empty(x[0].shape, dtype=BF, device="cuda"), torch.empty(x[1].shape, dtype=BF, device="cuda")]
    tfm.rope_rows(x[0], x[1], *out_rows, positions, dinv, interleaved=False, mscale=ms)
    tfm.cache8_write(out_rows[1], x[2], *cache, _ints(lens), block, cu_seqlens=_ends(new))
    torch.cuda.synchronize()
    follow(x, positions, lens, new)
    for T in (1, 3):
        x = torch.empty(B * T, H + 2 * Hkv, dh, dtype=BF, device="cuda")
        parts = x.split((H, Hkv, Hkv), 1)
        out_rows = [torch.empty(parts[0].shape, dtype=BF, device="cuda"), torch.empty(parts[1].shape, dtype=BF, device="cuda")]
        o = torch.empty(B * T, H, dh, dtype=BF, device="cuda")
        positions, dl = _ints([0] * (B * T)), _ints([0] * B)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            tfm.rope_rows(parts[0], parts[1], *out_rows, positions, dinv, interleaved=False, mscale=ms)
            tfm.cache8_write(out_rows[1], parts[2], *cache, dl, block)
            tfm.cache8_attention(out_rows[0], *cache, o, dl, ws, block, window=window)
        for step in range(8):
            lens = [n + T for n in lens]
            x.copy_(torch.randn(x.shape, generator=g) * (1 + step))
            positions.copy_(_ints([n - T + t for n in lens for t in range(T)]))
            dl.copy_(_ints(lens))
            graph.replay()
            torch.cuda.synchronize()
            follow(parts, positions, lens, [T] * B, o)
            lens = [n - (step % T) for n in lens]             # the last ones refused
    tfm.device_status()
