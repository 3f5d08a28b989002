"""Attention over packed prompts on the GPU (tfm_packed_attention) against its
plain form in 64 bits: lengths of zero and one, around the tiles' edges, grouped
heads, windows, layouts; rows of no sequence untouched; NaN and infinities in
places that a row does not see; offsets that are out of range; graphs, streams."""
import numpy as np
import pytest

from batch_ref import bound, f64, packed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


def _inputs(seed, T, H, Hkv, dh, dtype=torch.bfloat16, layout="token"):
    g = torch.Generator().manual_seed(seed)

    def rows(heads):
        if layout == "head":
            return torch.randn(heads, T, dh, generator=g).to(dtype).cuda().transpose(0, 1)
        return torch.randn(T, heads, dh, generator=g).to(dtype).cuda()

    if layout == "fused":
        x = torch.randn(T, H + 2 * Hkv, dh, generator=g).to(dtype).cuda()
        return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    return rows(H), rows(Hkv), rows(Hkv)


def _cu(lens, first=0):
    return torch.tensor([first] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _ws(T, n):
    return torch.empty(tfm.packed_attention_workspace_bytes(T, n), dtype=torch.uint8, device="cuda")


def _call(q, k, v, cu, window=0, scale=0.0, o=None):
    o = torch.full_like(q, 7.0, memory_format=torch.contiguous_format) if o is None else o
    tfm.packed_attention(q, k, v, o, cu, _ws(q.shape[0], cu.shape[0] - 1), window=window, scale=scale)
    torch.cuda.synchronize()
    return o


def _smax(q, k, scale):
    """The largest scaled sum of magnitudes a score can have."""
    a = f64(q.reshape(-1, q.shape[-1])) ** 2
    b = f64(k.reshape(-1, k.shape[-1])) ** 2
    return float(np.sqrt(np.nanmax(a.sum(-1)) * np.nanmax(b.sum(-1)))) * scale


def _check(o, q, k, v, lens, window=0, scale=None):
    n = sum(lens)
    dh = q.shape[-1]
    ref = packed(q[:n], k[:n], v[:n], lens, window, scale)
    tol = bound(f64(v[:n]), dh, max(lens, default=0), _smax(q[:n], k[:n], scale or dh ** -0.5), q.dtype) if n else 0
    got = f64(o[:n])
    assert np.isfinite(got).all()
    assert np.abs(got - ref).max(initial=0.0) <= tol
    assert (o[n:] == 7.0).all()                        # rows behind the last sequence


LENS = [[1], [5], [128], [129], [0, 5, 0, 128, 1, 0, 255, 256, 257, 0], [300, 0, 700, 3], [64, 64, 64], [1] * 40]


@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (3, 1)])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[:10])))
def test_lengths_and_heads(lens, H, Hkv, dh):
    T = sum(lens) + 9
    q, k, v = _inputs(dh + H + T, T, H, Hkv, dh)
    _check(_call(q, k, v, _cu(lens)), q, k, v, lens)


@pytest.mark.parametrize("dh", [4, 16, 64, 100, 128])
@pytest.mark.parametrize("lens", [[1, 0, 65, 130], [33, 64, 1], [200]], ids=str)
@pytest.mark.parametrize("window", [0, 40])
def test_fp32(lens, dh, window):
    T = sum(lens) + 3
    q, k, v = _inputs(dh + T, T, 4, 2, dh, torch.float32)
    _check(_call(q, k, v, _cu(lens), window), q, k, v, lens, window)


@pytest.mark.parametrize("dh,H,Hkv", [(32, 4, 4), (64, 6, 2), (128, 4, 1), (128, 2, 2)])
@pytest.mark.parametrize("window", [1, 2, 127, 128, 129, 200, 5000])
def test_windows(window, dh, H, Hkv):
    lens = [300, 1, 129, 0, 520]
    q, k, v = _inputs(window + dh, sum(lens) + 2, H, Hkv, dh)
    _check(_call(q, k, v, _cu(lens), window), q, k, v, lens, window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["head", "fused"])
@pytest.mark.parametrize("dh,H,Hkv", [(64, 4, 2), (128, 3, 3), (32, 8, 1)])
def test_layouts(layout, dh, H, Hkv, dtype):
    lens = [130, 7, 260]
    T = sum(lens) + 5
    q, k, v = _inputs(dh, T, H, Hkv, dh, dtype, layout)
    o = torch.full((H, T, dh), 7.0, dtype=dtype, device="cuda").transpose(0, 1)   # head-major output
    _check(_call(q, k, v, _cu(lens), o=o), q, k, v, lens)
    wide = torch.full((T, H, dh + 8), 7.0, dtype=dtype, device="cuda")           # padded output rows
    _check(_call(q, k, v, _cu(lens), o=wide[..., :dh]), q, k, v, lens)
    assert (wide[..., dh:] == 7.0).all()


def test_scale_and_large_scores():
    lens = [150, 30]
    q, k, v = _inputs(3, 180, 4, 4, 64)
    _check(_call(q, k, v, _cu(lens), scale=0.31), q, k, v, lens, scale=0.31)
    # Scores of several hundred: one key takes nearly all the weight and the running maximum moves
    # often.  Powers of two and few nonzero coordinates keep every score exact in fp32.
    q2, k2 = torch.zeros_like(q), torch.zeros_like(k)
    q2[..., 0], q2[..., 1] = 16.0, 8.0
    i = torch.arange(180, device="cuda")
    k2[..., 0] = ((i * 37) % 61).to(k.dtype)[:, None]
    k2[..., 1] = ((i * 11) % 13).to(k.dtype)[:, None]
    o = _call(q2, k2, v, _cu(lens), scale=1.0)
    ref = packed(q2, k2, v, lens, scale=1.0)
    tol = ((1 + 2.0 ** -8) ** 2 * (1 + 2.0 ** -12) - 1) * float(v.abs().max())
    assert np.abs(f64(o) - ref).max() <= tol


@pytest.mark.parametrize("dh,Hkv", [(32, 4), (64, 4), (128, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_sequences_are_not_seen(bad, dh, Hkv):
    """One sequence and the rows behind the last one hold nothing but `bad`: the others' rows keep their values."""
    lens = [70, 200, 33, 128, 1]
    T = sum(lens) + 20
    q, k, v = _inputs(dh, T, 4, Hkv, dh)
    for window in (0, 50):
        clean = _call(q, k, v, _cu(lens), window)
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for t in (q2, k2, v2):
            t[70:270] = bad
            t[432:] = bad
        o = _call(q2, k2, v2, _cu(lens), window)
        assert torch.equal(o[:70], clean[:70]) and torch.equal(o[270:], clean[270:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dh", [32, 64, 128])
def test_keys_behind_a_row_are_not_seen(dh, bad, dtype):
    """A value that is not finite reaches the rows that see it, in its own column, and no other; a key that is
    not finite reaches no row before it."""
    lens, at = [300, 40], 201
    q, k, v = _inputs(dh + 1, 340, 4, 2, dh, dtype)
    clean = _call(q, k, v, _cu(lens))
    v2 = v.clone()
    v2[at, 0, 3] = bad
    o = _call(q, k, v2, _cu(lens))
    same = torch.ones_like(o, dtype=torch.bool)
    same[at:300, :2, 3] = False                        # heads 0 and 1 read kv head 0
    assert torch.equal(o[same], clean[same])
    assert not torch.isfinite(o[~same]).any()
    o = _call(q, k, v2, _cu(lens), 30)                 # a row past the window does not see it either
    clean_w = _call(q, k, v, _cu(lens), 30)
    same[:] = True
    same[at:at + 30, :2, 3] = False
    assert torch.equal(o[same], clean_w[same])
    assert not torch.isfinite(o[~same]).any()
    k2 = k.clone()
    k2[at, 1] = float("nan")
    o = _call(q, k2, v, _cu(lens))
    assert torch.equal(o[:at], clean[:at]) and torch.equal(o[300:], clean[300:])
    assert torch.equal(o[:, :2], clean[:, :2])


def test_offsets_out_of_range_are_skipped():
    q, k, v = _inputs(5, 200, 4, 4, 64)
    ok = _call(q, k, v, _cu([50, 60]))
    for cu in ([0, 50, 20, 110], [0, 50, 300], [-5, 50], [0, 50, -1], [0, 50, 2 ** 31 - 1, 60], [100, 50]):
        o = _call(q, k, v, torch.tensor(cu, dtype=torch.int32).cuda())
        with pytest.raises(tfm.TfmError) as e:
            tfm.device_status()
        assert e.value.status == tfm.TFM_EINVAL
        if cu[:2] == [0, 50]:
            assert torch.equal(o[:50], ok[:50]) or cu[2] == 20
        assert (o[110:] == 7.0).all()
    o = _call(q, k, v, _cu([30, 40], first=20))        # rows before the first sequence stay
    assert (o[:20] == 7.0).all() and (o[90:] == 7.0).all() and (o[20:90] != 7.0).any()
    tfm.device_status()
    for cu in ([0], [0, 0], [0, 0, 0]):
        assert (_call(q, k, v, torch.tensor(cu, dtype=torch.int32).cuda()) == 7.0).all()


def test_repeated_calls_agree_and_graph_replays_new_lengths():
    q, k, v = _inputs(8, 900, 8, 2, 128)
    cu, ws, o = _cu([400, 500]), _ws(900, 2), torch.zeros(900, 8, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tfm.packed_attention(q, k, v, o, cu, ws)
        s.synchronize()
        first = o.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tfm.packed_attention(q, k, v, o, cu, ws)
            tfm.packed_attention(o, k, v, q2 := torch.zeros_like(o), cu, ws)   # the same workspace, one behind the other
    for lens in ([400, 500], [1, 899], [900, 0], [129, 128]):
        cu.copy_(_cu(lens))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        _check(o, q, k, v, lens)
        again = _call(o.clone(), k, v, cu, o=torch.zeros_like(o))
        assert torch.equal(again[:sum(lens)], q2[:sum(lens)])
        if lens == [400, 500]:
            assert torch.equal(o, first)


def test_many_sequences_and_a_long_one():
    lens = [3] * 700 + [4000] + [17] * 300
    q, k, v = _inputs(13, sum(lens), 2, 1, 64)
    o = _call(q, k, v, _cu(lens))
    a, n = 2100, 4000
    few = [lens[0]] * 700
    _check(torch.cat([o[:2100], torch.full_like(o[:1], 7.0)]), q[:2100], k[:2100], v[:2100], few)
    _check(o[a:a + n], q[a:a + n], k[a:a + n], v[a:a + n], [n])
    _check(o[a + n:], q[a + n:], k[a + n:], v[a + n:], [17] * 300)


MANY = [0, 5, 0, 128, 1, 0, 255, 257, 700, 64, 1300, 2, 127, 0]


@pytest.mark.parametrize("dh,H,Hkv", [(32, 32, 16), (64, 24, 24), (64, 48, 8), (128, 24, 12), (128, 21, 21)])
@pytest.mark.parametrize("window", [0, 1, 100, 320])
def test_more_items_than_ctas(window, dh, H, Hkv):
    """Several items per CTA, taken from the list, of one and of two query tiles."""
    T = sum(MANY) + 3
    q, k, v = _inputs(dh + H + window, T, H, Hkv, dh)
    o = _call(q, k, v, _cu(MANY), window)
    _check(o, q, k, v, MANY, window)
    assert torch.equal(_call(q, k, v, _cu(MANY), window), o)


@pytest.mark.parametrize("dh,H,Hkv", [(64, 24, 24), (128, 24, 12)])
def test_list_and_no_list_agree(dh, H, Hkv):
    """The first sequences alone, without a list, and among many: the same bits, as an item's own work is the same."""
    T = sum(MANY)
    q, k, v = _inputs(dh, T, H, Hkv, dh)
    n = sum(MANY[:4])
    few = [t[:n].contiguous() for t in (q, k, v)]
    assert torch.equal(_call(*few, _cu(MANY[:4])), _call(q, k, v, _cu(MANY))[:n])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 70])
def test_values_that_are_not_finite_among_many_items(window, bad):
    q, k, v = _inputs(3, sum(MANY), 24, 12, 128)
    clean = _call(q, k, v, _cu(MANY), window)
    start = np.cumsum([0] + MANY)
    v2, seen = v.clone(), torch.zeros_like(clean, dtype=torch.bool)
    for b, L in enumerate(MANY):                        # in every sequence, another kv head and column
        if L > 1:
            at, g, c = int(start[b]) + L // 2, b % 12, 7 * b % 128
            v2[at, g, c] = bad
            end = int(start[b + 1]) if window == 0 else min(int(start[b + 1]), at + window)
            seen[at:end, 2 * g:2 * g + 2, c] = True
    o = _call(q, k, v2, _cu(MANY), window)
    assert torch.equal(o[~seen], clean[~seen])
    assert not torch.isfinite(o[seen]).any()


def test_offsets_out_of_range_among_many():
    q, k, v = _inputs(15, 2000, 48, 24, 64)
    lens = [300, 500, 64, 700]
    ok = _call(q, k, v, _cu(lens))
    for cu in ([0, 300, 800, 400, 1564], [0, 300, 800, 864, 2 ** 31 - 1], [-7, 300, 800, 864, 1564]):
        o = _call(q, k, v, torch.tensor(cu, dtype=torch.int32).cuda())
        with pytest.raises(tfm.TfmError) as e:
            tfm.device_status()
        assert e.value.status == tfm.TFM_EINVAL
        if cu[1:3] == [300, 800] and cu[3] == 864:
            assert torch.equal(o[300:864], ok[300:864])
        assert (o[1600:] == 7.0).all()
