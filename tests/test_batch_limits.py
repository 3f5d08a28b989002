"""Limits of the batched-serving entry points as the header states them, on both sides: what is beyond is refused by name;
what is not gets past that check, to the one for the pointers, which are NULL here.  No GPU is touched."""
import ctypes

import pytest

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


def test_verification_workspace_limit(lib):
    V = 1 << 24
    each = 8 * 2048 + 16 * 4096 + 32 + 4                 # statistics, candidates, decision, counter of a sequence
    most = (1 << 33) // each
    for B, ok in ((most - 4, True), (most + 4, False)):
        n = lib.tfm_verify_draft_workspace_bytes(B, 0, V)
        assert (0 < n < 1 << 33) if ok else n == 0
        assert ("NULL pointer" if ok else "2^33 bytes") in _verify(lib, B, 0, V)
