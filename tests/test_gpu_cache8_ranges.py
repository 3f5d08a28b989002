"""The 8-bit cache's operators on the GPU at the ends of their ranges, against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402
from test_gpu_cache8_attention import _cache, _call, _check, _q, _with_room  # noqa: E402

BF, I8, E4 = torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("H,Hkv,T,dh", [(8, 2, 1, 64), (8, 2, 3, 128), (10, 2, 4, 128), (8, 1, 4, 32)])
@pytest.mark.parametrize("scale,q_size,k_size", [
    (2.0 ** 120, -123, 0), (2.0 ** 126, -126, -3), (2.0 ** 126, -130, 1), (2.0 ** 126, 0, -126), (0.0, -124, 124), (0.0, 120, -119),
    (2.0 ** -13, 125, -115), (2.0 ** -100, 110, -13), (2.0 ** -140, 125, 12), (2.0 ** 60, -120, 57)], ids=str)
def test_scores_whose_factors_are_far_apart(scale, q_size, k_size, H, Hkv, T, dh, codes):
    """scale, q and the keys' scales near the ends of fp32, their product of ordinary size; a row of zeros among the others sees
    the mean of V.  The weights' and values' tolerances are those of ordinary factors: a power of two in each changes nothing
    but the range.  In a small cache (8 rows a job) and in one with room (up to 32 rows)."""
    lens, block = [200, 333], 16
    cache = _cache(31, 2, Hkv, 336, dh, block, codes)
    cache[2].mul_(2.0 ** k_size)
    q = (_q(31, 2 * T, H, dh).float() * 2.0 ** q_size).to(BF)
    q[1 % (2 * T), H - 1] = 0.0
    q[0, 0] = 0.0
    for c in (cache, _with_room(cache, block, 128 * (152 * 16 * 3 // 2 // (2 * Hkv) + 4))):
        o = _call(q, c, lens, block, scale=scale)
        _check(o, q, cache, lens, block, [T, T], 0, scale or None)


def test_no_kv_heads():
    """Hkv = 0: k and k_out are not used, whatever they point to."""
    import ctypes
    q = _q(51, 9, 4, 64)
    inv, pos = tfm.rope_frequencies(10000.0, 64)[0].cuda(), torch.arange(9, dtype=torch.int32, device="cuda")
    want, o = torch.zeros_like(q), torch.zeros_like(q)
    tfm.rope_rows(q, None, want, None, pos, inv)
    odd, strides = ctypes.c_void_p(257), (ctypes.c_int64 * 8)(256, 64, 0, -5, 256, 64, 0, 1 << 60)
    status = tfm.load().tfm_rope_rows(q.data_ptr(), odd, o.data_ptr(), odd, pos.data_ptr(), inv.data_ptr(), 9, 4, 0, 64, 64, 1,
                                      strides, 1.0, tfm.TFM_BF16, torch.cuda.current_stream().cuda_stream)
    assert status == tfm.TFM_OK, tfm.load().tfm_last_error()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("B,n,H,Hkv,dh", [(64, 4096, 8, 8, 64), (128, 8192, 8, 8, 32), (40, 4096, 64, 8, 128), (40, 4096, 128, 8, 128),
                                          (40, 4096, 192, 8, 64), (40, 4096, 256, 8, 128)])
def test_values_that_cancel_over_long_runs(B, n, H, Hkv, dh, codes):
    """Scores are equal, and every other tile holds the codes of the one before with the other sign, at the same scale: what a
    warp adds up is x, 0, x, 0 ..  Inside a step sums are of whole multiples of 2^-17 (int8: products up to 255 2^7 2^-24, and the
    bias of 16 times 128 of them) or 2^-2 (e4m3), fewer than 2^24 of them: exact in any order.  So an output is zero but for the
    tiles that a cut leaves without the other one: two parts, or four of a warp each, of at most 127 steps of one tile in n / 64,
    in 8 roundings of 2^-24: below 2^-19 of a step of the code for 64 tiles, and 2^-17 is asked for."""
    g = torch.Generator(device="cuda").manual_seed(dh)
    c = torch.randint(-127, 128, (B, Hkv, n // 128, 1, 64, dh), generator=g, device="cuda", dtype=torch.int8).float()
    if codes == E4:
        c = (c / 16).round()                                  # up to 8: exact
    cache = [torch.zeros(B, Hkv, n, dh, dtype=torch.int8, device="cuda").view(codes),
             torch.cat([c, -c], 3).view(B, Hkv, n, dh).to(codes),
             *((1 + torch.rand(B, Hkv, n // 128, generator=g, device="cuda")) / 50 for _ in "kv")]
    q = torch.randn(B, H, dh, generator=g, device="cuda").to(BF)
    o = _call(q, cache, [n] * B, 128)
    step = cache[3].amax(-1)[:, :, None].expand(B, Hkv, H // Hkv).reshape(B, H, 1)
    worst = float((o.float().abs() / step).max())
    assert worst <= 2.0 ** -17, np.log2(worst)


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("size", [120, 116, 112, 100, 64, -60, -100, -115])
def test_values_of_any_size(size, codes):
    """Values of up to 2^125 and down to 2^-126: the mean of values is no larger than the largest, and it comes out as precise
    as any, whether jobs are cut or whole, in jobs of 8 and of up to 32 rows, over thousands of positions, and where the
    running maximum lags behind (the weights are then 2^15)."""
    for lens, H, Hkv, T, dh, block, window, room in (
            ([1, 5], 8, 2, 1, 64, 16, 0, 0), ([200, 333], 8, 2, 3, 128, 16, 0, 0), ([20000, 70], 8, 1, 1, 64, 128, 0, 0),
            ([3000, 1], 4, 4, 1, 32, 16, 100, 0), ([256, 130], 16, 2, 2, 128, 32, 0, 300000), ([256, 130], 10, 2, 4, 128, 32, 0, 300000),
            ([256, 130], 8, 1, 4, 64, 32, 0, 300000)):
        n = 256 if room else max(lens) + 3
        cache = _cache(41, 2, Hkv, n, dh, block, codes)
        cache[3].mul_(2.0 ** size)
        q = _q(41, 2 * T, H, dh)
        wide = _with_room(cache, block, room // block * block) if room else cache
        _check(_call(q, wide, lens, block, window=window), q, cache, lens, block, [T, T], window)
        # the first 16 scores are 0, all others 5.4 (7.8 in powers of two)
        cache[0].zero_(), cache[2].fill_(2.0 ** -4)
        cache[0][:, :, 16:, 0] = 64.0 if codes == E4 else 64
        q.zero_()
        q[:, :, 0] = 1.35
        wide = _with_room(cache, block, room // block * block) if room else cache
        _check(_call(q, wide, lens, block, window=window, scale=1.0), q, cache, lens, block, [T, T], window, 1.0)


@pytest.mark.parametrize("codes", [I8, E4])
def test_values_of_one_block_far_above_the_others(codes):
    """Blocks of 2^110 and 2^120 among ordinary ones, early, late and between, in small and in cut jobs; rows that see none of
    them, beside rows that do, have the precision of ordinary ones."""
    for lens, H, Hkv, T, dh in (([200, 337], 8, 2, 3, 128), ([20000, 17], 8, 1, 1, 64), ([337, 49], 4, 2, 8, 32)):
        for where in (slice(0, 1), slice(2, 4), slice(11, 12), slice(15, 22), slice(0, 1 << 20)):
            for far in (2.0 ** 70, 2.0 ** 110, 2.0 ** 120):
                cache = _cache(43, 2, Hkv, max(lens) + 3, dh, 16, codes)
                cache[3][:, :, where] *= far
                q = _q(43, 2 * T, H, dh)
                _check(_call(q, cache, lens, 16), q, cache, lens, 16, [T, T])
    # the last of T tokens begins a block of its own
    for T, H, Hkv in ((2, 8, 2), (4, 8, 2), (8, 16, 4)):
        lens, block = [97, 337], 16
        cache = _cache(44, 2, Hkv, 340, 64, block, codes)
        for b, n in enumerate(lens):
            cache[3][b, :, n // block] = 2.0 ** 118
        q = _q(44, 2 * T, H, 64)
        o = _call(q, cache, lens, block)
        _check(o, q, cache, lens, block, [T, T])
        before, qb = (x.view(2, T, H, 64)[:, :-1].reshape(-1, H, 64) for x in (o, q))
        _check(before, qb, cache, [n - 1 for n in lens], block, [T - 1, T - 1])


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_an_infinity_among_zeros(dtype, codes):
    """A block without a finite value but zeros has the scale 0 and the code 0 for the infinity too: when a later token gives the
    block a scale, it stays 0, as all values that a block holds stay what they are."""
    for bad in (float("inf"), -float("inf"), float("nan")):
        kc, vc, ks, vs = _cache(52, 1, 2, 64, 64, 32, codes)
        k = torch.zeros(20, 2, 64, dtype=dtype, device="cuda")
        k[7, 1, 3] = bad
        for rows, n in ((k, 20), (torch.ones(1, 2, 64, dtype=dtype, device="cuda"), 21)):
            tfm.cache8_write(rows, rows, kc, vc, ks, vs, torch.tensor([n], dtype=torch.int32, device="cuda"), 32)
            torch.cuda.synchronize()
            if n == 20:
                with pytest.raises(tfm.TfmError) as e:
                    tfm.device_status()
                assert e.value.status == tfm.TFM_EINVAL
                assert (ks[:, :, 0] == 0).all() and (vs[:, :, 0] == 0).all()
            for c in (kc, vc):
                assert (c.float()[:, :, :20] == 0).all()
        tfm.device_status()
        top = 127 if codes == I8 else 448.0
        assert (kc.float()[:, :, 20] == top).all() and (ks[:, :, 0] == (torch.ones(1) / top).cuda()).all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,Hkv,dh,rot", [(1, 5, 5, 20, 20), (7, 3, 1, 20, 20), (300, 5, 5, 20, 20), (4000, 3, 3, 20, 20),
                                            (2000, 3, 2, 36, 12), (3000, 3, 3, 10, 2), (500, 7, 1, 6, 2)])
def test_rotations_behind_one_another_as_calls_apart(T, H, Hkv, dh, rot, interleaved):
    """In place, where rows of neighbouring tokens and heads share a sector of memory, at accesses of 8, 4 and 2 bytes: the bits
    of the same calls with the device waited for in between."""
    g = torch.Generator().manual_seed(T)
    rows = torch.randn(T, H + Hkv, dh, generator=g).to(BF).cuda()
    inv = tfm.rope_frequencies(10000.0, rot)[0].cuda()
    positions = [torch.randint(-1000, 1000, (T,), generator=g, dtype=torch.int32).cuda() for _ in range(12)]

    def rotate(x, wait):
        q, k = x.split((H, Hkv), 1)
        for p in positions:
            tfm.rope_rows(q, k, q, k, p, inv, interleaved=interleaved)
            if wait:
                torch.cuda.synchronize()

    want = rows.clone()
    rotate(want, True)
    x = rows.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        rotate(x, False)
    for recorded in (False, True, True, True):
        x.copy_(rows)
        torch.cuda.synchronize()
        if recorded:
            graph.replay()
        else:
            rotate(x, False)
        torch.cuda.synchronize()
        assert torch.equal(x.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("H,Hkv,T,room", [(4, 4, 1, 0), (8, 2, 2, 0), (10, 2, 4, 300000)])
def test_rows_of_q_that_are_not_finite(H, Hkv, T, room, codes):
    """They come out NaN, whatever the keys are (with every key's score minus infinity too); a row that sees nothing is zero."""
    lens, block = [200, 70, 0], 32
    cache = _cache(53, 3, Hkv, 224, 64, block, codes)
    cache[0][:, :, :, 5] = torch.tensor(-3.0).to(codes).item()
    wide = _with_room(cache, block, room // block * block) if room else cache
    q = _q(53, 3 * T, H, 64)
    clean = _call(q, wide, lens, block)
    for bad in (float("inf"), -float("inf"), float("nan")):
        x = q.clone().view(3, T, H, 64)
        x[:, T - 1, 1, 5] = bad
        o = _call(x.view(3 * T, H, 64), wide, lens, block).view(3, T, H, 64)
        assert o[:2, T - 1, 1].isnan().all() and (o[2] == 0).all()
        same = torch.ones(3, T, H, dtype=torch.bool, device="cuda")
        same[:2, T - 1, 1] = False
        assert torch.equal(o[same], clean.view(3, T, H, 64)[same])


@pytest.mark.parametrize("codes", [I8, E4])
@pytest.mark.parametrize("lens,H,Hkv,T,dh,block,window,room", [
    ([200, 337], 8, 2, 1, 128, 16, 0, 0), ([20000, 70], 8, 1, 1, 64, 16, 0, 0), ([5000, 4000, 64], 4, 2, 2, 32, 128, 0, 0),
    ([30000], 8, 1, 1, 128, 128, 0, 0), ([3000, 2999], 4, 4, 1, 64, 32, 700, 0), ([384, 130], 10, 2, 4, 128, 32, 0, 300000),
    ([384, 200], 16, 2, 2, 64, 16, 0, 300000), ([384, 384], 8, 1, 4, 128, 16, 0, 300000)], ids=lambda x: str(x)[:20])
def test_values_on_both_sides_of_the_larger_units(lens, H, Hkv, T, dh, block, window, room, codes):
    """Scales of V of 2^63 and 2^64, and a few of 1.5 2^64, which some warps and pieces of a job meet and others do not (the sums
    of those that do are in units of 2^64): a part taken for the other kind would be 2^64 off."""
    n = -(-max(lens) // 128) * 128
    for seed, often in ((0, 0.5), (1, 0.05), (2, 0.005), (3, 0.0)):
        cache = _cache(45 + seed, len(lens), Hkv, n, dh, block, codes)
        g = torch.Generator().manual_seed(seed)
        pick = torch.rand(cache[3].shape, generator=g)
        cache[3].copy_(torch.where(pick < often, 1.5 * 2.0 ** 64, torch.where(pick < 0.75, 2.0 ** 64, 2.0 ** 63)))
        if often == 0.0:                                       # one block alone, the last whole one of the first sequence
            cache[3][0, :, max(lens[0] // block - 1, 0)] = 1.5 * 2.0 ** 64
        q = _q(45, len(lens) * T, H, dh)
        wide = _with_room(cache, block, room // block * block) if room else cache
        _check(_call(q, wide, lens, block, window=window), q, cache, lens, block, [T] * len(lens), window)
