"""Attention over a shared prefix and own caches on the GPU (tfm_prefix_attention)
against its plain form in 64 bits."""
import numpy as np
import pytest

from batch_ref import bound, f64, prefix

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


def _inputs(seed, B, H, Hkv, T, P, room, dh):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    return r(B, H, T, dh), r(Hkv, P, dh), r(Hkv, P, dh), r(B, Hkv, room, dh), r(B, Hkv, room, dh)


def _lens(lens):
    return torch.tensor(lens, dtype=torch.int32).cuda()


def _call(q, kp, vp, kc, vc, lens, prefix_len=None, scale=0.0):
    B, H, T, dh = q.shape
    ws = torch.empty(tfm.prefix_attention_workspace_bytes(B, H, kc.shape[1], T, dh), dtype=torch.uint8, device="cuda")
    o = torch.full((B, T, H * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    tfm.prefix_attention(q, kp, vp, kc, vc, o, lens, ws, prefix_len=prefix_len, scale=scale)
    torch.cuda.synchronize()
    return o


def _check(o, q, kp, vp, kc, vc, lens, P=None, scale=None):
    P = kp.shape[1] if P is None else P
    dh = q.shape[-1]
    ref = prefix(q, kp, vp, kc, vc, lens, P, scale)
    norm = lambda t: float(np.sqrt((f64(t) ** 2).sum(-1).max(initial=0.0)))
    smax = norm(q) * max(norm(kp[:, :P]), norm(kc)) * (scale or dh ** -0.5)
    v = np.concatenate([f64(vp[:, :P]).ravel(), f64(vc).ravel()])
    got = f64(o)
    assert np.isfinite(got).all()
    assert np.abs(got - ref).max() <= bound(v, dh, P + max(lens), smax, torch.bfloat16)


@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("H,Hkv,T", [(4, 4, 1), (8, 2, 1), (8, 1, 1), (6, 2, 5), (4, 4, 3), (16, 1, 8), (3, 3, 128)])
@pytest.mark.parametrize("P,lens", [(1, [1]), (300, [1, 64, 65, 0, 200]), (128, [7, 128, 129]), (64, [0, 0]),
                                    (1000, [130] * 19), (0, [5, 1, 300])], ids=str)
def test_sizes(P, lens, H, Hkv, T, dh):
    lens = [n + (T - 1 if n else 0) for n in lens]
    a = _inputs(P + T + dh, len(lens), H, Hkv, T, max(P, 1), max(lens) + 3, dh)
    _check(_call(*a, _lens(lens), P), *a, lens, P)


@pytest.mark.parametrize("T", [1, 4])
def test_empty_rows_and_short_caches(T):
    """Without prefix: a token that sees no key gets zeros; caches shorter than T."""
    a = _inputs(4, 4, 4, 2, T, 5, 9, 64)
    lens = [0, 1, 2, 9]
    o = _call(*a, _lens(lens), 0)
    _check(o, *a, lens, 0)
    assert (o[0] == 0).all()
    _check(_call(*a, _lens(lens), 5), *a, lens, 5)


def test_what_lies_behind_the_lengths_is_not_looked_at():
    lens = [3, 70, 0, 64, 130]
    for T in (1, 3):
        q, kp, vp, kc, vc = _inputs(T, 5, 8, 2, T, 200, 140, 128)
        lens_t = _lens(lens)
        clean = _call(q, kp, vp, kc, vc, lens_t, 150)
        for bad in (float("nan"), float("inf"), -3e38):
            kp2, vp2, kc2, vc2 = kp.clone(), vp.clone(), kc.clone(), vc.clone()
            for t in (kp2, vp2):
                t[:, 150:] = bad
            for t in (kc2, vc2):
                for b, n in enumerate(lens):
                    t[b, :, n:] = bad
            assert torch.equal(_call(q, kp2, vp2, kc2, vc2, lens_t, 150), clean)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_drafted_tokens_do_not_see_those_behind_them(bad):
    q, kp, vp, kc, vc = _inputs(7, 3, 4, 2, 4, 100, 80, 64)
    lens = [80, 5, 64]
    clean = _call(q, kp, vp, kc, vc, _lens(lens))
    for back in (1, 2, 3):                              # the new token T - back .. T - 1 sees it
        vc2, kc2 = vc.clone(), kc.clone()
        for b, n in enumerate(lens):
            vc2[b, 1, n - back, 5] = bad
            kc2[b, 0, n - back] = float("nan")
        o = _call(q, kp, vp, kc, vc2, _lens(lens)).view(3, 4, 4, 64)
        same = torch.ones_like(o, dtype=torch.bool)
        same[:, 4 - back:, 2:, 5] = False
        assert torch.equal(o[same], clean.view(3, 4, 4, 64)[same])
        assert not torch.isfinite(o[~same]).any()
        o = _call(q, kp, vp, kc2, vc, _lens(lens)).view(3, 4, 4, 64)
        assert torch.equal(o[:, :4 - back], clean.view(3, 4, 4, 64)[:, :4 - back])
        assert torch.equal(o[:, :, 2:], clean.view(3, 4, 4, 64)[:, :, 2:])


def test_one_sequence_does_not_reach_another():
    lens = [100, 40, 257]
    q, kp, vp, kc, vc = _inputs(9, 3, 4, 4, 1, 300, 300, 64)
    clean = _call(q, kp, vp, kc, vc, _lens(lens))
    for t in (q, kc, vc):
        t[1] = float("nan")
    o = _call(q, kp, vp, kc, vc, _lens(lens))
    assert torch.equal(o[0], clean[0]) and torch.equal(o[2], clean[2])


def test_decode_attention_agrees_without_a_prefix():
    """T = 1 and no prefix is tfm_decode_attention at each sequence's own length: the same bf16 answer up to two
    roundings of weights and outputs on each side."""
    q, kp, vp, kc, vc = _inputs(11, 4, 8, 4, 1, 1, 333, 64)
    o = _call(q, kp, vp, kc, vc, _lens([333] * 4), 0)
    ws = torch.empty(tfm.decode_attention_workspace_bytes(4, 8, 333, 64), dtype=torch.uint8, device="cuda")
    d = torch.empty(4, 512, dtype=torch.bfloat16, device="cuda")
    tfm.decode_attention(q.view(4, 8, 64), kc, vc, d, 332, ws)
    torch.cuda.synchronize()
    assert float((o.view(4, 512).float() - d.float()).abs().max()) <= 4.2 * 2.0 ** -8 * float(vc.abs().max())


def test_lengths_out_of_range_count_as_zero():
    a = _inputs(2, 3, 4, 2, 1, 50, 40, 64)
    o = _call(*a, _lens([41, -1, 40]))
    with pytest.raises(tfm.TfmError) as e:
        tfm.device_status()
    assert e.value.status == tfm.TFM_EINVAL
    _check(o, *a, [0, 0, 40])


def test_scale_and_graph_with_new_lengths():
    a = _inputs(6, 5, 8, 2, 2, 500, 400, 128)
    lens = _lens([5, 100, 400, 2, 77])
    _check(_call(*a, lens, 300, 0.2), *a, [5, 100, 400, 2, 77], 300, 0.2)
    ws = torch.empty(tfm.prefix_attention_workspace_bytes(5, 8, 2, 2, 128), dtype=torch.uint8, device="cuda")
    o = torch.zeros(5, 2, 1024, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tfm.prefix_attention(*a, o, lens, ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tfm.prefix_attention(*a, o, lens, ws)
    for new in ([5, 100, 400, 2, 77], [400] * 5, [0, 2, 0, 399, 64], [0] * 5):
        lens.copy_(_lens(new))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        _check(o, *a, new)
        assert torch.equal(o, _call(*a, lens))


def test_large_batch():
    lens = [(i * 37) % 90 + 1 for i in range(600)]
    a = _inputs(12, 600, 4, 2, 1, 700, 91, 32)
    _check(_call(*a, _lens(lens)), *a, lens)
