"""Rotary positions of packed rows on the GPU (tfm_rope_rows) against the rotation in 64 bits."""
import numpy as np
import pytest

from batch_ref import f64
from cache8_ref import rope

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


def _rows(seed, T, *heads, dh, dtype=BF, fused=False):
    g = torch.Generator().manual_seed(seed)
    if fused:
        return torch.randn(T, sum(heads), dh, generator=g).to(dtype).cuda().split(heads, 1)
    return [torch.randn(T, h, dh, generator=g).to(dtype).cuda() for h in heads]


def _close(got, x, positions, inv, interleaved, mscale):
    """Sine and cosine: the fraction of a turn rounded to 2^-25 of a turn (1.9e-7 in the angle), the functions themselves
    within 2 ulp, the factor: 9 roundings of 2^-24; two products and a sum: 3 more.  The turns per position are held to
    2^-51 of themselves and 2^-62.  The value is rounded to its type."""
    want, size = rope(x, positions.tolist(), inv.tolist(), interleaved, mscale)
    pos = np.abs(f64(positions))[:, None, None]
    far = pos * (float(inv.abs().max()) * 2.0 ** -50 + 2.0 ** -60)
    tol = size * (12 * 2.0 ** -24 + far) + np.abs(want) * torch.finfo(got.dtype).eps / 2 * 1.001 + 1e-38
    r = 2 * len(inv)
    assert (np.abs(f64(got) - want)[..., :r] <= tol[..., :r]).all()
    assert torch.equal(got[..., r:], x[..., r:])


def _call(q, k, positions, inv, interleaved=True, mscale=1.0):
    qo, ko = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), None if k is None else torch.full(k.shape, 7.0, dtype=k.dtype, device="cuda")
    tfm.rope_rows(q, k, qo, ko, positions, inv, interleaved=interleaved, mscale=mscale)
    torch.cuda.synchronize()
    return qo, ko


def _pos(seed, T, far=100000):
    return torch.randint(0, far, (T,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,Hkv,dh,rot", [
    (1, 16, 4, 128, 128), (1, 1, 1, 2, 2), (5, 12, 12, 64, 16), (33, 3, 1, 80, 40), (17, 2, 2, 20, 20), (7, 5, 1, 6, 4),
    (130, 16, 4, 128, 64), (64, 4, 4, 16, 16), (9, 2, 1, 256, 256), (3, 3, 3, 31, 30), (6, 2, 2, 96, 8), (2, 40, 8, 128, 32),
    (5000, 2, 1, 32, 32), (11, 7, 3, 66, 64)])
def test_sizes(T, H, Hkv, dh, rot, dtype, interleaved):
    q, k = _rows(T + rot, T, H, Hkv, dh=dh, dtype=dtype)
    inv, _ = tfm.rope_frequencies(10000.0, rot)
    pos = _pos(T, T)
    for mscale in (1.0, 1.277):
        qo, ko = _call(q, k, pos, inv.cuda(), interleaved, mscale)
        _close(qo, q, pos, inv, interleaved, float(np.float32(mscale)))
        _close(ko, k, pos, inv, interleaved, float(np.float32(mscale)))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("shift", [0, 1])
def test_fused_projection_in_place_and_unaligned(interleaved, shift):
    """Columns of one projection, head-major rows, rows that start between two 16-byte marks; in place as out of place,
    and nothing beside the rows is written."""
    inv, _ = tfm.rope_frequencies(500000.0, 32, "wavelength", factor=8.0, original=512, low=1.0, high=4.0)
    inv, pos = inv.cuda(), _pos(1, 37)
    around = torch.randn(37 * 9 * 64 + 8, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    x = around[shift:shift + 37 * 9 * 64].view(37, 9, 64)
    q, k, v = x.split((4, 2, 3), 1)
    qo, ko = _call(q, k, pos, inv, interleaved)
    _close(qo, q, pos, inv.cpu(), interleaved, 1.0)
    _close(ko, k, pos, inv.cpu(), interleaved, 1.0)
    before = around.clone()
    tfm.rope_rows(q, k, q, k, pos, inv, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(q[..., 32:], before[shift:shift + 37 * 9 * 64].view(37, 9, 64)[:, :4, 32:])
    assert torch.equal(v, before[shift:shift + 37 * 9 * 64].view(37, 9, 64)[:, 6:])
    assert torch.equal(around[:shift], before[:shift]) and torch.equal(around[shift + 37 * 9 * 64:], before[shift + 37 * 9 * 64:])
    heads = torch.randn(4, 37, 64, generator=torch.Generator().manual_seed(4)).to(BF).cuda().transpose(0, 1)
    qo, none = _call(heads, None, pos, inv, interleaved)
    assert none is None
    _close(qo, heads, pos, inv.cpu(), interleaved, 1.0)


def test_far_and_negative_positions():
    """Every int32 position: the angle is reduced exactly."""
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 24 + 1, -2 ** 24 - 3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    q, k = _rows(5, 8, 2, 1, dh=128, dtype=F32)
    for inv in (tfm.rope_frequencies(10000.0, 128)[0], torch.tensor([3.0, -0.7, 6.5, 0.0, 1e-9, 100.25], dtype=torch.float64)):
        for interleaved in (True, False):
            qo, ko = _call(q, k, pos, inv.cuda(), interleaved)
            _close(qo, q, pos, inv, interleaved, 1.0)
            _close(ko, k, pos, inv, interleaved, 1.0)
    assert torch.equal(qo[0], q[0])                                  # position 0 turns nothing


def test_rope_of_the_heads_agrees():
    """tfm_rope on [B, H, S, dh] is the same rotation: each side rounds once, the angles agree to fp32."""
    x = torch.randn(2, 3, 50, 64, generator=torch.Generator().manual_seed(6)).cuda()
    pos = _pos(7, 100, 5000)
    rows = x.permute(0, 2, 1, 3).reshape(100, 3, 64)
    qo, _ = _call(rows, None, pos, tfm.rope_frequencies(10000.0, 64)[0].cuda())
    tfm.rope(x, 10000.0, pos.view(2, 50))
    torch.cuda.synchronize()
    assert float((qo.view(2, 50, 3, 64).permute(0, 2, 1, 3) - x).abs().max()) <= 24 * 2.0 ** -24 * 2 * float(x.abs().max())


def test_rotation_is_undone_by_the_opposite_positions():
    q, k = _rows(8, 300, 4, 2, dh=64, dtype=F32)
    inv, pos = tfm.rope_frequencies(10000.0, 64)[0].cuda(), _pos(8, 300)
    back, kb = _call(*_call(q, k, pos, inv, False), -pos, inv, False)
    assert float((back - q).abs().max()) <= 2 * 2 * 12 * 2.0 ** -24 * 2 * float(q.abs().max())


def test_values_that_are_not_finite_stay_in_their_pair():
    q, k = _rows(9, 20, 4, 2, dh=64)
    inv, pos = tfm.rope_frequencies(10000.0, 64)[0].cuda(), _pos(9, 20)
    for interleaved, pair in ((True, [10, 11]), (False, [10, 42])):
        clean, kc = _call(q, k, pos, inv, interleaved)
        bad = q.clone()
        bad[3, 1, 10] = float("nan")
        o, kb = _call(bad, k, pos, inv, interleaved)
        same = torch.ones_like(o, dtype=torch.bool)
        same[3, 1, pair] = False
        assert torch.equal(o[same], clean[same]) and o[~same].isnan().all() and torch.equal(kb, kc)


def test_graph_stream_and_empty():
    q, k = _rows(10, 40, 16, 4, dh=128)
    inv, pos = tfm.rope_frequencies(10000.0, 128)[0].cuda(), _pos(10, 40)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tfm.rope_rows(q, k, qo, ko, pos, inv)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tfm.rope_rows(q, k, qo, ko, pos, inv)
    for i in range(3):
        pos.copy_(_pos(20 + i, 40))
        g.replay()
        torch.cuda.synchronize()
        want, kw = _call(q, k, pos, inv)
        assert torch.equal(qo, want) and torch.equal(ko, kw)
    e = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    tfm.rope_rows(e, None, e, None, torch.empty(0, dtype=torch.int32, device="cuda"), inv[:8])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("start", [2, 4, 8])
@pytest.mark.parametrize("T,H,Hkv,dh,rot", [(9, 3, 2, 80, 40), (700, 2, 1, 80, 40), (6, 5, 0, 256, 256), (40, 1, 3, 36, 12), (3, 4, 4, 254, 4)])
def test_rows_that_start_between_16_byte_marks(T, H, Hkv, dh, rot, start, dtype, interleaved):
    """Accesses of 4, 8 and 16 bytes; what lies around the rows stays."""
    heads = H + Hkv
    wide = torch.randn(T, heads * dh + 24, generator=torch.Generator().manual_seed(T)).to(dtype).cuda()
    out = torch.full_like(wide, 7.0)
    inv, _ = tfm.rope_frequencies(10000.0, rot)
    pos = _pos(T, T)
    parts = lambda x: x[:, start:start + heads * dh].unflatten(1, (heads, dh)).split((H, Hkv), 1)
    (q, k), (qo, ko) = parts(wide), parts(out)
    if not Hkv:
        k = ko = None
    tfm.rope_rows(q, k, qo, ko, pos, inv.cuda(), interleaved=interleaved)
    torch.cuda.synchronize()
    _close(qo, q, pos, inv, interleaved, 1.0)
    if Hkv:
        _close(ko, k, pos, inv, interleaved, 1.0)
    assert (out[:, :start] == 7.0).all() and (out[:, start + heads * dh:] == 7.0).all()
