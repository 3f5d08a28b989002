"""Writing the 8-bit cache and reading it back on the GPU (tfm_cache8_write, tfm_cache8_read):
codes, scales and values have to be those of 64 bits."""
import numpy as np
import pytest

from batch_ref import f64
from cache8_ref import TOP, code, write

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402

BF, F32, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


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


def _cache(seed, B, Hkv, room, dh, block, dtype):
    """k and v codes and scales as earlier writes left them (every code and a scale near 0.02)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in "kv":
        c = torch.randint(-127, 128, (B, Hkv, room, dh), generator=g)
        out.append((c.to(torch.int8) if dtype == I8 else torch.where(c == 0, c, c).to(torch.int8).view(E4)).cuda())
    if dtype == E4:
        for c in out:                                        # 0x7f and 0xff are NaN, which a write never stores
            c.view(torch.uint8)[(c.view(torch.uint8) & 127) == 127] = 0
    top = TOP[dtype]
    s = [(torch.rand(B, Hkv, -(-room // block), generator=g) * 2 + 1).cuda() / top for _ in "kv"]
    return [*out, *s]


def _rows(seed, T, Hkv, dh, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(T, Hkv, dh, generator=g) * std).to(dtype).cuda() for _ in "kv"]


def _written(cache, k, v, lens, new, block, cu=True, status=None):
    """The cache after the call, which has to be what 64 bits say, bit for bit."""
    kc, vc, ks, vs = (t.clone() for t in cache)
    dtype = kc.dtype
    want = [write(x, f64(c.float()), f64(s), lens, new, block, dtype) for x, c, s in ((k, kc, ks), (v, vc, vs))]
    tfm.cache8_write(k, v, kc, vc, ks, vs, _ints(lens), block, cu_seqlens=_ends(new) if cu else None)
    torch.cuda.synchronize()
    if status is None:
        tfm.device_status()
    else:
        with pytest.raises(tfm.TfmError) as e:
            tfm.device_status()
        assert e.value.status == status
    for (c, s), gc, gs in zip(want, (kc, vc), (ks, vs)):
        assert np.array_equal(f64(gs), s)
        assert np.array_equal(f64(gc.float()), c)
    return kc, vc, ks, vs


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,dh", [(1, 32), (3, 64), (4, 128)])
@pytest.mark.parametrize("lens,new", [
    ([1], [1]), ([300], [300]), ([300, 1, 0, 17, 128, 64], [300, 1, 0, 17, 128, 64]),
    ([65, 64, 16, 129, 1, 300, 33], [1, 1, 1, 1, 1, 1, 1]), ([70, 5, 128, 200], [5, 0, 3, 140])], ids=str)
def test_codes_and_scales(lens, new, Hkv, dh, block, dtype, codes):
    cache = _cache(block + dh, len(lens), Hkv, 307, dh, block, codes)
    for std in (0.3, 3.0):                                   # below most of the scales that are there, and above
        k, v = _rows(sum(new), sum(new), Hkv, dh, dtype, std)
        _written(cache, k, v, lens, new, block)


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quotients_on_and_beside_the_borders_between_codes(codes, dtype):
    """Rows made of (code + half a step) * scale, a rounding of the input to either side, for scales of every size, those
    too small or large for a reciprocal among them."""
    top = TOP[codes]
    vals = np.arange(0, 127.0) + 0.5 if codes == I8 else np.unique(np.abs(code(np.linspace(0, 448, 20001), E4)))
    if codes == E4:
        vals = (vals[1:] + vals[:-1]) / 2
    rng = np.random.default_rng(5)
    for e in (-126, -120, -101, -60, -3, 0, 1, 50, 99, 100, 118):
        blocks = []
        for _ in range(4):
            amax = np.float32(2.0 ** e * (1 + rng.integers(0, 128) / 128) * (top if e < 110 else 1))
            if dtype == BF:
                amax = f64(torch.tensor(float(amax)).to(BF))[()]
            s = float(np.float32(amax / top))
            x = np.zeros(16 * 64, np.float32)
            m = np.float32(rng.choice(vals, 16 * 64) * s)
            x[:] = m
            x[::3], x[1::3] = np.nextafter(m[::3], np.float32(0)), np.nextafter(m[1::3], np.float32(np.inf))
            x *= rng.choice([-1, 1], x.size)
            x = np.clip(x, -amax, amax).astype(np.float32)
            x[0] = amax
            blocks.append(x.reshape(16, 1, 64))
        x = torch.from_numpy(np.concatenate(blocks)).to(dtype).cuda()
        cache = _cache(1, 1, 1, 64, 64, 16, codes)
        _written(cache, x, -x, [64], [64], 16)


@pytest.mark.parametrize("codes", [I8, E4])
def test_a_scale_that_grows_token_by_token(codes):
    """One token at a time, sizes rising and falling over 40 powers of two: codes and scales at every step, and what is
    left of the first token: off by a step of the scale at most beyond its own rounding."""
    block, dh, n = 32, 32, 64
    cache = _cache(3, 2, 2, n, dh, block, codes)
    g = torch.Generator().manual_seed(8)
    size = torch.exp2(torch.randint(-20, 21, (n,), generator=g).float())
    rows = [(torch.randn(n, 2, 2, dh, generator=g) * size[:, None, None, None]).to(BF).cuda() for _ in "kv"]
    for t in range(n):
        k, v = (r[t].contiguous() for r in rows)
        cache = _written(cache, k, v, [t + 1, t + 1], [1, 1], block, cu=t % 2 == 0)
    kept = f64(cache[0].float())[0, 0] * np.repeat(f64(cache[2])[0, 0], block)[:, None]
    exact, scale = f64(rows[0][:, 0, 0]), np.repeat(f64(cache[2])[0, 0], block)[:, None]
    step = scale if codes == I8 else np.maximum(np.abs(exact) / 8, scale * 2.0 ** -9)
    assert (np.abs(kept - exact) <= 1.5 * step).all()


@pytest.mark.parametrize("codes", [I8, E4])
def test_zeros_and_cut_back_sequences(codes):
    block = 16
    cache = _cache(4, 1, 1, 64, 32, block, codes)
    z = torch.zeros(20, 1, 32, dtype=BF, device="cuda")
    cache = _written(cache, z, z, [20], [20], block)                     # scale 0
    k, v = _rows(1, 3, 1, 32, BF)
    cache = _written(cache, k, v, [23], [3], block)                      # joins a block of scale 0
    k, v = _rows(2, 5, 1, 32, BF, 9.0)
    cache = _written(cache, k, v, [26], [5], block)                      # two of the three tokens are taken back
    k, v = _rows(3, 1, 1, 32, BF, 0.01)
    cache = _written(cache, k, v, [17], [1], block)                      # a block of which nothing is left
    _written(cache, k, v, [1], [1], block)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_that_are_not_finite(bad, codes, dtype):
    cache = _cache(6, 3, 2, 90, 64, 32, codes)
    k, v = _rows(4, 120, 2, 64, dtype)
    k[50, 1, 7] = bad
    v[119] = bad
    out = _written(cache, k, v, [60, 45, 40], [60, 45, 15], 32, status=tfm.TFM_EINVAL)
    assert np.isfinite(f64(out[2])).all() and np.isfinite(f64(out[0].float())).all()


@pytest.mark.parametrize("lens,cu", [([41, 5], [0, 10, 15]), ([-1, 5], [0, 10, 15]), ([9, 5], [0, 10, 15]),
                                     ([20, 5], [0, 10, 16]), ([20, 5], [0, 10, 9]), ([20, 5], [-1, 10, 15]),
                                     ([20, 20], [0, 2 ** 31 - 1, 15]), ([20, 20], [-2 ** 31, 2, 15])], ids=str)
def test_lengths_and_offsets_out_of_range(lens, cu):
    """The error word says so; the sequence is not written (or read), nor anything around the buffers."""
    whole = _cache(7, 4, 2, 40, 32, 16, I8)
    kept = [t.clone() for t in whole]
    inner = [t[1:3] for t in whole]
    k, v = _rows(5, 15, 2, 32, BF)
    for read in (False, True):
        if read:
            tfm.cache8_read(*inner, k, v, _ints(lens), 16, cu_seqlens=_ints(cu))
        else:
            tfm.cache8_write(k, v, *inner, _ints(lens), 16, cu_seqlens=_ints(cu))
        with pytest.raises(tfm.TfmError) as e:
            tfm.device_status()
        assert e.value.status == tfm.TFM_EINVAL
    for a, b in zip(whole, kept):
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[3].view(torch.uint8), b[3].view(torch.uint8))
    ok = [0 <= cu[b] <= cu[b + 1] <= 15 and cu[b + 1] - cu[b] <= lens[b] <= 40 for b in range(2)]
    for b in range(2):
        if not ok[b]:
            assert all(torch.equal(a[1 + b], c[1 + b]) for a, c in zip(whole, kept))


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,Hkv,dh", [(16, 3, 32), (64, 2, 64), (128, 4, 128)])
def test_reading_back(block, Hkv, dh, dtype, codes):
    """The values are fp32 products rounded once; any part of the end of a sequence; strided rows; nothing else written."""
    lens, new = [300, 0, 17, 128, 64, 1], [300, 0, 5, 100, 64, 1]
    kc, vc, ks, vs = _cache(9, 6, Hkv, 301, dh, block, codes)
    T = sum(new) + 4
    x = torch.full((T, 2 * Hkv + 1, dh), 7.0, dtype=dtype, device="cuda")
    k, _, v = x.split((Hkv, 1, Hkv), 1)
    tfm.cache8_read(kc, vc, ks, vs, k, v, _ints(lens), block, cu_seqlens=_ends(new))
    torch.cuda.synchronize()
    tfm.device_status()
    for got, c, s in ((k, kc, ks), (v, vc, vs)):
        want = (c.float().cpu() * s.cpu().repeat_interleave(block, 2)[:, :, :301, None]).to(dtype)
        rows = torch.cat([want[b, :, L - n:L].transpose(0, 1) for b, (L, n) in enumerate(zip(lens, new))])
        assert torch.equal(got[:sum(new)].cpu(), rows)
    assert (x[sum(new):] == 7.0).all() and (x[:, Hkv] == 7.0).all()


@pytest.mark.parametrize("codes", [I8, E4])
def test_round_trip_is_half_a_step_off(codes):
    k, v = _rows(11, 500, 4, 128, F32)
    cache = _cache(2, 2, 4, 400, 128, 64, codes)
    out = _written(cache, k, v, [380, 120], [380, 120], 64)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    tfm.cache8_read(*out, ko, vo, _ints([380, 120]), 64, cu_seqlens=_ends([380, 120]))
    for x, y, s in ((k, ko, out[2]), (v, vo, out[3])):
        top = s[:2].amax().item()
        half = torch.full_like(x, top / 2) if codes == I8 else (x.abs() * 2.0 ** -4).clamp(min=top * 2.0 ** -10)
        assert ((x - y).abs() <= half * (1 + 1e-5)).all()


def test_fused_rows_streams_and_graph():
    """Rows that are columns of one projection, the cache of more sequences than the batch, a recorded graph with new
    lengths."""
    block, Hkv, dh = 32, 2, 64
    x = torch.randn(6, 8, dh, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    _, k, v = x.split((4, 2, 2), 1)
    cache = _cache(5, 9, Hkv, 100, dh, block, I8)
    lens = _ints([1, 40, 100])
    live = [t.clone() for t in cache]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tfm.cache8_write(k, v, *live, lens, block)
    for new in ([2, 40, 100], [33, 65, 2], [50, 51, 52]):
        for a, b in zip(live, cache):
            a.copy_(b)
        lens.copy_(_ints(new))
        g.replay()
        torch.cuda.synchronize()
        small = [t[:3] for t in cache]
        want = _written(small, k.contiguous(), v.contiguous(), new, [2, 2, 2], block, cu=False)
        for a, b, c in zip(live, want, cache):
            assert torch.equal(a[:3], b) and torch.equal(a[3:], c[3:])


def test_many_sequences():
    """Sequences are found among thousands of offsets, empty ones in a row too."""
    rng = np.random.default_rng(3)
    new = np.where(rng.random(4096) < 0.3, 0, rng.integers(1, 40, 4096)).tolist()
    lens = [n + int(e) for n, e in zip(new, rng.integers(0, 20, 4096))]
    cache = _cache(12, 4096, 1, 64, 32, 16, I8)
    k, v = _rows(13, sum(new), 1, 32, BF)
    _written(cache, k, v, lens, new, 16)


def test_offsets_beyond_32_bits():
    """The last positions of a cache of more than 2^32 codes."""
    room, block = 4_400_001, 128
    kc, vc = (torch.empty(2, 4, room, 128, dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(2, 4, -(-room // block), device="cuda") for _ in "kv")
    k, v = _rows(14, 300, 4, 128, BF)
    lens, new = _ints([130, room]), _ends([130, 170])
    tfm.cache8_write(k, v, kc, vc, ks, vs, lens, block, cu_seqlens=new)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    tfm.cache8_read(kc, vc, ks, vs, ko, vo, lens, block, cu_seqlens=new)
    torch.cuda.synchronize()
    tfm.device_status()
    first = (room - 170) // block * block
    small = [torch.zeros(2, 4, 512, 128, dtype=torch.int8, device="cuda") for _ in "kv"] + [torch.zeros(2, 4, 4, device="cuda") for _ in "kv"]
    tfm.cache8_write(k, v, *small, _ints([130, room - first]), block, cu_seqlens=new)
    ks2, vs2 = torch.zeros_like(k), torch.zeros_like(v)
    tfm.cache8_read(*small, ks2, vs2, _ints([130, room - first]), block, cu_seqlens=new)
    assert torch.equal(ko, ks2) and torch.equal(vo, vs2) and float((ko - k).abs().max()) < 0.05


@pytest.mark.parametrize("B", [31, 32, 33, 63, 64, 65, 94, 95, 96, 97])
@pytest.mark.parametrize("block,dh", [(16, 32), (64, 64), (128, 128)])
def test_numbers_of_sequences(B, block, dh):
    """Up to 32, up to 95 and more of them are found in different ways; warps that share a unit, and those that do not."""
    rng = np.random.default_rng(B)
    new = np.where(rng.random(B) < 0.3, 0, rng.integers(1, 150, B)).tolist()
    new[-1] = 3 if B % 2 else 0
    lens = [n + int(e) for n, e in zip(new, rng.integers(0, 60, B))]
    cache = _cache(B, B, 2, 210, dh, block, I8)
    k, v = _rows(B + 1, sum(new) + 2, 2, dh, BF)
    kc, vc, ks, vs = _written(cache, k, v, lens, new, block)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    tfm.cache8_read(kc, vc, ks, vs, ko, vo, _ints(lens), block, cu_seqlens=_ends(new))
    torch.cuda.synchronize()
    tfm.device_status()
    for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
        want = (c.float().cpu() * s.cpu().repeat_interleave(block, 2)[:, :, :210, None]).to(BF)
        assert torch.equal(got[:sum(new)].cpu(), torch.cat([want[b, :, L - n:L].transpose(0, 1) for b, (L, n) in enumerate(zip(lens, new))]))
        assert (got[sum(new):] == 7.0).all()


@pytest.mark.parametrize("bad", [2 ** 31 - 1, -2 ** 31, -1, 301])
@pytest.mark.parametrize("B,block", [(33, 16), (64, 128), (95, 64)])
def test_an_offset_out_of_range_among_many(B, block, bad):
    """The two sequences that it bounds are left as they were, and what lies around the buffers."""
    whole = _cache(7, B + 2, 2, 40, 64, block, I8)
    kept = [t.clone() for t in whole]
    inner = [t[1:B + 1] for t in whole]
    new = [3] * B
    k, v = _rows(5, 300, 2, 64, BF)
    cu = _ends(new)
    cu[20] = bad
    for read in (False, True):
        f = tfm.cache8_read if read else tfm.cache8_write
        args = (*inner, k, v) if read else (k, v, *inner)
        f(*args, _ints([20] * B), block, cu_seqlens=cu)
        with pytest.raises(tfm.TfmError) as e:
            tfm.device_status()
        assert e.value.status == tfm.TFM_EINVAL
    for a, b in zip(whole, kept):
        for i in (0, 20, 21, B + 1):
            assert torch.equal(a[i].view(torch.uint8), b[i].view(torch.uint8))
