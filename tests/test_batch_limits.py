"""Limits of the batched-serving entry points as the header states them, on both sides: what is beyond is refused by name;
what is not gets past that check, to the one for the pointers, which are NULL here.  No GPU is touched."""
import numpy as np
import pytest
import torch

from decoder_only_transformer_gb300 import tfm


@pytest.fixture(scope="module")
def lib():
    return tfm.load()


def _prefix(lib, B, H, Hkv, T, P, max_seq, dh=64, scale=0.0):
    st = lib.tfm_prefix_attention(None, None, None, None, None, None, None, B, H, Hkv, T, P, P, max_seq, dh, scale, None, 0, None)
    assert st == tfm.TFM_EINVAL
    return lib.tfm_last_error().decode()


def _verify(lib, B, K, V):
    ld = (V + 3) // 4 * 4
    st = lib.tfm_verify_draft(None, ld, None, ld, None, None, None, None, ld, B, K, V, 1.0, None, None, None, 0, None)
    assert st == tfm.TFM_EINVAL
    return lib.tfm_last_error().decode()


@pytest.mark.parametrize("B,H,Hkv,T,P,max_seq", [
    (1, 1, 1, 1, ((1 << 25) - 1) * 64, 64),              # the prefix alone, but for one tile
    (4096, 4096, 4096, 1, 128 * 64, 63),                 # own caches of a tile each, the prefix 32 times
    (1, 100, 1, 1, 64, 1),
    (4096, 2, 1, 1, 1 << 20, 1 << 16),
])
def test_prefix_key_tiles(lib, B, H, Hkv, T, P, max_seq):
    nb = 128 // (H // Hkv * T)
    tiles = lambda p: Hkv * -(-B // nb) * -(-p // 64) + B * Hkv * -(-max_seq // 64)
    assert tiles(P) <= 1 << 25
    assert "NULL pointer" in _prefix(lib, B, H, Hkv, T, P, max_seq)
    if tiles(P + 1) > 1 << 25:
        assert "key tiles" in _prefix(lib, B, H, Hkv, T, P + 1, max_seq)


@pytest.mark.parametrize("B,H,Hkv,T,P", [(1, 1, 1, 1, (1 << 31) - 1), (1, 1, 1, 1, (1 << 31) - 63), (4096, 100, 1, 1, 1 << 20),
                                         (2, 128, 128, 64, (1 << 24) - 1)])
def test_prefix_beyond_its_key_tiles(lib, B, H, Hkv, T, P):
    assert "key tiles" in _prefix(lib, B, H, Hkv, T, P, 1)


@pytest.mark.parametrize("scale,ok", [(2.0 ** 126, True), (2.0 ** 126 * (1 + 2.0 ** -23), False), (3.4e38, False), (1e-45, True),
                                      (-3.4e38, True), (float("inf"), False)])
def test_scales_that_the_kernels_can_apply(lib, scale, ok):
    want = "NULL pointer" if ok else "scale"
    assert want in _prefix(lib, 1, 1, 1, 1, 1, 1, scale=scale)
    for mode in (tfm.TFM_BF16, tfm.TFM_FP32):
        assert lib.tfm_packed_attention(None, None, None, None, None, 1, 4, 1, 1, 64, None, scale, 0, mode, None, 0, None) == tfm.TFM_EINVAL
        assert want in lib.tfm_last_error().decode()


def test_verification_workspace_limit(lib):
    V = 1 << 24
    each = 8 * 2048 + 16 * 4096 + 32 + 4                 # statistics, candidates, decision, counter of a sequence
    most = (1 << 33) // each
    for B, ok in ((most - 4, True), (most + 4, False)):
        n = lib.tfm_verify_draft_workspace_bytes(B, 0, V)
        assert (0 < n < 1 << 33) if ok else n == 0
        assert ("NULL pointer" if ok else "2^33 bytes") in _verify(lib, B, 0, V)


class _Cuda:
    """As much of a dense tensor on device 0 as the binding looks at, of any size."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.is_cuda, self.device = tuple(shape), dtype, True, torch.device("cuda:0")
        self.nbytes = 1 << 62

    def stride(self, i=None):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * max(n, 1))
        return tuple(s) if i is None else s[i]

    def numel(self):
        return int(np.prod([int(n) for n in self.shape], dtype=object))

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256


BIG = (1 << 32) + 5                                      # 5 in its low bits


@pytest.fixture
def no_library(monkeypatch):
    """No call reaches the library: what it was given is returned."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or 0

    monkeypatch.setattr(tfm, "_lib", Lib())
    monkeypatch.setattr(tfm, "_now", lambda: (torch, 0))
    monkeypatch.setattr(tfm, "_raw_stream", lambda stream, device: 0)
    return calls


def _packed_call(T=8, H=2, Hkv=2, n=1, **kw):
    bf, ints = torch.bfloat16, torch.int32
    q, kv = (T, H, 32), (T, Hkv, 32)
    tfm.packed_attention(_Cuda(q, bf), _Cuda(kv, bf), _Cuda(kv, bf), _Cuda(q, bf), _Cuda((n + 1,), ints), _Cuda((64,), torch.uint8), **kw)


def _prefix_call(B=2, H=2, T=1, P=8, cap=2, rows=8, **kw):
    bf = torch.bfloat16
    p, c = (2, P, 32), (cap, 2, rows, 32)
    tfm.prefix_attention(_Cuda((B, H, T, 32), bf), _Cuda(p, bf), _Cuda(p, bf), _Cuda(c, bf), _Cuda(c, bf),
                         _Cuda((B, T, H * 32), bf), _Cuda((B,), torch.int32), _Cuda((64,), torch.uint8), **kw)


def _verify_call(B=2, K=2, V=8, vocab=8, **kw):
    f, i = torch.float32, torch.int32
    tfm.verify_draft(_Cuda((B * (K + 1), V), f), _Cuda((B * K, V), f), _Cuda((B, K), i), None, _Cuda((B, K), f), _Cuda((B, V), f),
                     vocab, _Cuda((B, K + 1), i), _Cuda((B,), i), _Cuda((64,), torch.uint8), **kw)


@pytest.mark.parametrize("call,kw", [
    (_packed_call, dict(T=BIG)), (_packed_call, dict(H=BIG, Hkv=1)), (_packed_call, dict(H=BIG, Hkv=BIG)),
    (_packed_call, dict(n=BIG)), (_packed_call, dict(window=BIG)), (_packed_call, dict(window=-BIG)),
    (_prefix_call, dict(B=BIG, cap=BIG)), (_prefix_call, dict(T=BIG)), (_prefix_call, dict(P=BIG)), (_prefix_call, dict(rows=BIG)),
    (_prefix_call, dict(prefix_len=BIG)), (_prefix_call, dict(prefix_len=-BIG)),
    (_verify_call, dict(B=BIG)), (_verify_call, dict(V=BIG, vocab=BIG)), (_verify_call, dict(V=BIG, vocab=BIG, temperature=0.0)),
], ids=str)
def test_numbers_beyond_32_bits_are_refused(no_library, call, kw):
    call()
    assert len(no_library) == 1                          # the call is otherwise in order
    with pytest.raises(ValueError, match="32 bits"):
        call(**kw)
    assert len(no_library) == 1


@pytest.mark.parametrize("size", [lambda n: tfm.packed_attention_workspace_bytes(n, 1), lambda n: tfm.packed_attention_workspace_bytes(1, n),
                                  lambda n: tfm.prefix_attention_workspace_bytes(n, 1, 1, 1, 64),
                                  lambda n: tfm.verify_draft_workspace_bytes(1, 1, n)])
def test_workspaces_of_numbers_beyond_32_bits(size):
    assert size(5) > 0
    with pytest.raises(ValueError, match="32 bits"):
        size(BIG)
