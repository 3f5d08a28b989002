"""Calls of the batched-serving operators that lie at the edge of what their documentation allows."""
import numpy as np
import pytest

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


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _packed(q, k, v, cu, **kw):
    o = torch.full_like(q, 7.0)
    tfm.packed_attention(q, k, v, o, cu, _bytes(tfm.packed_attention_workspace_bytes(len(q), len(cu) - 1)), **kw)
    torch.cuda.synchronize()
    return o


@pytest.mark.parametrize("H,Hkv,dh", [(1, 1, 32), (3, 1, 64), (2, 1, 32)])
def test_a_value_that_is_not_finite_in_every_prompt(H, Hkv, dh):
    """Thousands of items, twenty and more per CTA, with and without a second query tile, each with an infinity at its
    last key: only the row of that key sees it."""
    rng = np.random.default_rng(H * dh)
    lens = np.where(rng.random(3600 // H) < 0.2, rng.integers(129, 300, 3600 // H), rng.integers(1, 129, 3600 // H))
    cu = np.concatenate([[0], np.cumsum(lens)])
    g = torch.Generator().manual_seed(dh)
    q, k, v = (torch.randn(int(cu[-1]), h, dh, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
    want = _packed(q, k, v, _ints(cu))
    last = torch.from_numpy(cu[1:] - 1).cuda()
    bad = v.clone()
    bad[last, :, 5] = float("inf")
    want[last, :, 5] = float("inf")
    for _ in range(5):
        assert torch.equal(_packed(q, k, bad, _ints(cu)), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu", [[0, 150, 20, 110], [0, 300, 50, 110], [0, 200, 0, 200, 0, 200], [-5, 70, 200], [10, 2 ** 31 - 1, -2 ** 31, 90],
                                [200, 150, 100, 50, 0], [0] + [190, 10] * 300], ids=lambda x: "-".join(map(str, x[:5])))
@pytest.mark.parametrize("H", [1, 40])                  # each block a CTA of its own, or a list
def test_offsets_that_decrease_or_leave_the_rows(cu, H, dtype):
    """The device error word says so, and nothing around the buffers is written."""
    T, dh = 200, 32
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(T, H, dh, generator=g).to(dtype).cuda() for _ in range(3))
    around = torch.full((3 * T, H, dh), 7.0, dtype=dtype, device="cuda")
    n = tfm.packed_attention_workspace_bytes(T, len(cu) - 1)
    ws = torch.full((3 * 4096 + n,), 99, dtype=torch.uint8, device="cuda")
    tfm.packed_attention(q, k, v, around[T:2 * T], _ints(cu), ws[4096:4096 + n])
    with pytest.raises(tfm.TfmError) as e:
        tfm.device_status()
    assert e.value.status == tfm.TFM_EINVAL
    assert (around[:T] == 7.0).all() and (around[2 * T:] == 7.0).all()
    assert (ws[:4096] == 99).all() and (ws[4096 + n:] == 99).all()
    # the next call with offsets as they should be is as ever
    want = _packed(q, k, v, _ints([0, 150, 200]))
    tfm.device_status()
    assert torch.isfinite(want).all()


def test_large_scores_in_fp32():
    """Scores of some hundreds: the scale folded with log2(e) and the approximate exponential stay within the roundings
    that the bound counts (it has 2 dh for the score, of which the product takes dh, the folded scale 2)."""
    from batch_ref import bound, f64, packed
    for dh, lens, factor, scale in ((16, [150, 31], 4.0, 1.7), (64, [200], 3.0, 0.0), (128, [97, 64], 2.0, 0.3), (4, [300], 8.0, 0.9)):
        g = torch.Generator().manual_seed(dh)
        q, k, v = (torch.randn(sum(lens), 2, dh, generator=g).cuda() * f for f in (factor, factor, 1.0))
        got = f64(_packed(q, k, v, _ints(np.cumsum([0] + lens)), scale=scale))
        s = float(np.float32(scale)) or dh ** -0.5
        norm = lambda t: float(np.sqrt((f64(t) ** 2).sum(-1).max()))
        smax = norm(q) * norm(k) * s
        assert smax > 100
        assert np.abs(got - packed(q, k, v, lens, 0, s)).max() <= bound(f64(v), dh, max(lens), smax, torch.float32)
