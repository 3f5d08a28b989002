"""Rows of the batched-serving attentions keep their bits whatever lies behind the keys they see: the rows of a prompt
when it grows by a few tokens, and any row when the values behind the last key it sees change.  A row maximum taken
over keys that are masked would not change a result beyond its roundings, only its bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402

LENS = [1, 31, 33, 37, 63, 64, 65, 100, 125, 128, 190, 300]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


def _rand(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def _packed(q, k, v, n, window):
    o = torch.zeros_like(q)
    ws = torch.empty(tfm.packed_attention_workspace_bytes(len(q), 1), dtype=torch.uint8, device="cuda")
    tfm.packed_attention(q, k, v, o, torch.tensor([0, n], dtype=torch.int32).cuda(), ws, window=window)
    return o[:n]


@pytest.mark.parametrize("dh,dtype", [(32, torch.bfloat16), (64, torch.bfloat16), (128, torch.bfloat16),
                                      (16, torch.float32), (64, torch.float32)], ids=str)
@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 3)])
@pytest.mark.parametrize("window", [0, 50])
def test_packed_rows(dh, dtype, H, Hkv, window):
    for n in LENS:
        g = torch.Generator().manual_seed(n + dh)
        m = n + 3
        q, k, v = _rand(g, m, H, dh, dtype=dtype), _rand(g, m, Hkv, dh, dtype=dtype), _rand(g, m, Hkv, dh, dtype=dtype)
        want = _packed(q[:n], k[:n], v[:n], n, window)
        assert torch.equal(_packed(q, k, v, m, window)[:n], want), n
        for factor in (0.0, 30.0):                     # rows of no sequence, in the same tiles
            a, b, c = q.clone(), k.clone(), v.clone()
            for t in (a, b, c):
                t[n:] *= factor
            assert torch.equal(_packed(a, b, c, n, window), want), n


def _prefix(q, kp, vp, kc, vc, lens, prefix_len):
    B, H, T, dh = q.shape
    o = torch.zeros(B, T, H * dh, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(tfm.prefix_attention_workspace_bytes(B, H, kc.shape[1], T, dh), dtype=torch.uint8, device="cuda")
    tfm.prefix_attention(q, kp, vp, kc, vc, o, torch.tensor(lens, dtype=torch.int32).cuda(), ws, prefix_len=prefix_len)
    return o


@pytest.mark.parametrize("dh", [32, 64, 128])
@pytest.mark.parametrize("H,Hkv,T", [(4, 4, 1), (8, 2, 3)])
@pytest.mark.parametrize("P", [0, 37, 500])
def test_what_lies_behind_a_cache(dh, H, Hkv, T, P):
    for n in LENS:
        g = torch.Generator().manual_seed(n + dh + P)
        lens, room = [n, max(n - 5, 0), n + 30], n + 70
        q, kc, vc = _rand(g, 3, H, T, dh), _rand(g, 3, Hkv, room, dh), _rand(g, 3, Hkv, room, dh)
        kp, vp = _rand(g, Hkv, P + 20, dh), _rand(g, Hkv, P + 20, dh)
        want = _prefix(q, kp, vp, kc, vc, lens, P)
        for factor in (0.0, 30.0):
            a, b, c, d = kp.clone(), vp.clone(), kc.clone(), vc.clone()
            for t in (a, b):
                t[:, P:] *= factor
            for t in (c, d):
                for i, m in enumerate(lens):
                    t[i, :, m:] *= factor
            assert torch.equal(_prefix(q, a, b, c, d, lens, P), want), n


@pytest.mark.parametrize("dh", [32, 64, 128])
def test_tokens_behind_a_token(dh):
    """The first of four new tokens sees what a single one with three positions fewer does (caches of up to two tiles of
    64 keys: one piece in either call)."""
    for n in LENS:
        if n > 125:
            continue
        g = torch.Generator().manual_seed(n + dh)
        q, kc, vc = _rand(g, 1, 4, 4, dh), _rand(g, 1, 4, n + 3, dh), _rand(g, 1, 4, n + 3, dh)
        none = torch.empty(4, 0, dh, dtype=torch.bfloat16, device="cuda")
        four = _prefix(q, none, none, kc, vc, [n + 3], 0)
        one = _prefix(q[:, :, :1].contiguous(), none, none, kc, vc, [n], 0)
        assert torch.equal(four[:, :1], one), n
