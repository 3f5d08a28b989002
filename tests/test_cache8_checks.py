"""Host-side checks of the 8-bit cache's entry points: every limit the header states is
refused before any pointer is read, empty calls return at once, workspace sizes, the
rotary frequencies, and the binding's refusals.  No GPU is touched; the pointers are
aligned but point nowhere."""
import ctypes
import math

import pytest
import torch

from decoder_only_transformer_gb300 import tfm

B16, F32 = tfm.TFM_BF16, tfm.TFM_FP32
E, U, OK = tfm.TFM_EINVAL, tfm.TFM_EUNSUPPORTED, tfm.TFM_OK
A = ctypes.c_void_p(256)
INF, NAN = float("inf"), float("nan")


def P(n):
    return ctypes.c_void_p(n)


@pytest.fixture(scope="module")
def lib():
    return tfm.load()


def _st(d, n):
    if d["strides"] is not None:
        d["strides"] = (ctypes.c_int64 * n)(*d["strides"])


def _rope(lib, **kw):
    d = dict(q=A, k=A, qo=P(512), ko=P(512), pos=A, inv=A, T=10, H=4, Hkv=2, dh=64, rot=64, inter=1, strides=None, ms=1.0,
             mode=B16)
    d.update(kw)
    _st(d, 8)
    return lib.tfm_rope_rows(*d.values(), None)


def _write(lib, read=False, **kw):
    d = dict(k=A, v=A, kc=A, vc=A, ks=A, vs=A, cu=A, lens=A, B=3, T=10, Hkv=2, dh=64, max_seq=100, block=16, strides=None,
             codes=0, mode=B16)
    d.update(kw)
    _st(d, 4)
    a = list(d.values())
    return lib.tfm_cache8_read(*a[2:6], *a[:2], *a[6:], None) if read else lib.tfm_cache8_write(*a, None)


def _read(lib, **kw):
    return _write(lib, True, **kw)


def _attend(lib, **kw):
    d = dict(q=A, kc=A, vc=A, ks=A, vs=A, o=A, cu=A, lens=A, B=3, T=10, H=4, Hkv=2, max_new=5, dh=64, max_seq=100, block=16,
             strides=None, codes=0, window=0, scale=0.0, ws=A, nbytes=1 << 30)
    d.update(kw)
    _st(d, 4)
    return lib.tfm_cache8_attention(*d.values(), None)


def _but(dense, i, v):
    s = list(dense)
    s[i] = v
    return s


ROPE = [256, 64, 128, 64, 256, 64, 128, 64]
ROWS = [128, 64, 128, 64]
Q = [256, 64, 256, 64]


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), E), (dict(T=(1 << 30) + 1), E), (dict(H=0), E), (dict(H=4097), E), (dict(Hkv=-1), E), (dict(Hkv=4097), E),
    (dict(dh=1), E), (dict(dh=257), E), (dict(rot=0), E), (dict(rot=63), E), (dict(rot=66), E), (dict(rot=-2), E),
    (dict(mode=7), E), (dict(ms=NAN), E), (dict(ms=INF), E),
    (dict(q=None), E), (dict(k=None), E), (dict(qo=None), E), (dict(ko=None), E), (dict(pos=None), E), (dict(inv=None), E),
    (dict(q=P(257)), E), (dict(ko=P(513)), E), (dict(q=P(258), mode=F32), E), (dict(pos=P(258)), E), (dict(inv=P(260)), E),
    (dict(strides=_but(ROPE, 0, 63)), E), (dict(strides=_but(ROPE, 3, -64)), E), (dict(strides=_but(ROPE, 6, 1 << 39)), E),
    (dict(qo=A, strides=_but(ROPE, 4, 512)), E),                 # in place at other strides
    (dict(ko=A, strides=_but(ROPE, 7, 72)), E),
    (dict(T=0), OK), (dict(T=0, q=None, k=None, qo=None, ko=None, pos=None, inv=None), OK), (dict(T=0, rot=3), E),
])
def test_rope_rows_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status, lib.tfm_last_error()
    if status != OK:
        assert lib.tfm_last_error()


CACHE = [
    (dict(B=-1), E), (dict(B=4097), E), (dict(T=-1), E), (dict(T=(1 << 30) + 1), E), (dict(Hkv=0), E), (dict(Hkv=4098), E),
    (dict(max_seq=0), E), (dict(B=4096, Hkv=4, max_seq=1 << 17), E), (dict(codes=2), E), (dict(codes=-1), E),
    (dict(dh=0), E), (dict(block=0), E), (dict(dh=48), U), (dict(dh=256), U), (dict(block=8), U), (dict(block=48), U),
    (dict(block=256), U), (dict(cu=None), E),                     # 10 rows of 3 sequences
    (dict(kc=None), E), (dict(vc=None), E), (dict(ks=None), E), (dict(vs=None), E), (dict(lens=None), E),
    (dict(kc=P(264)), E), (dict(vc=P(264)), E), (dict(ks=P(258)), E), (dict(vs=P(258)), E), (dict(lens=P(258)), E),
    (dict(cu=P(258)), E), (dict(B=0), OK), (dict(T=0), OK), (dict(B=0, kc=None, vc=None, ks=None, vs=None, lens=None), OK),
    (dict(T=0, dh=48), U), (dict(B=0, block=8), U),
]


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(mode=7), E), (dict(k=None), E), (dict(v=None), E), (dict(k=P(264)), E), (dict(v=P(258)), E),
    (dict(strides=_but(ROWS, 0, 63)), E), (dict(strides=_but(ROWS, 1, 68)), E), (dict(strides=_but(ROWS, 2, 1 << 39)), E),
    (dict(B=1, Hkv=4096, max_seq=1, T=1 << 22), E), (dict(B=1, Hkv=4096, max_seq=1, T=(1 << 22) - 64, k=None), E),   # units
    (dict(strides=_but(ROWS, 3, 0)), E), (dict(strides=_but(ROWS, 1, 66), mode=F32), E),
])
def test_write_and_read_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status, lib.tfm_last_error()
    if status != OK:
        assert lib.tfm_last_error()


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(H=0), E), (dict(H=5), E), (dict(max_new=0), E), (dict(B=4096, H=4096, Hkv=4096, max_seq=1, max_new=2), E),
    (dict(window=-1), E), (dict(scale=NAN), E), (dict(scale=INF), E), (dict(scale=1e38), E),
    (dict(max_new=65), U), (dict(H=256), U), (dict(cu=None, T=18), E),            # six rows each, max_new 5
    (dict(q=None), E), (dict(o=None), E), (dict(ws=None), E), (dict(q=P(264)), E), (dict(o=P(264)), E), (dict(ws=P(264)), E),
    (dict(strides=_but(Q, 0, 63)), E), (dict(strides=_but(Q, 1, 68)), E), (dict(strides=_but(Q, 2, 1 << 39)), E),
    (dict(nbytes=0), E),
])
def test_attention_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status, lib.tfm_last_error()
    if status != OK:
        assert lib.tfm_last_error()


def test_attention_workspace(lib):
    size = lib.tfm_cache8_attention_workspace_bytes
    n = size(3, 4, 2, 5, 64)
    assert n > 0 and _attend(lib, nbytes=n - 1) == E
    assert b"workspace too small" in lib.tfm_last_error()
    for bad in ((-1, 4, 2, 5, 64), (4097, 4, 2, 5, 64), (3, 5, 2, 5, 64), (3, 4, 2, 0, 64), (3, 4, 2, 65, 64), (3, 4, 2, 5, 48)):
        assert size(*bad) == 0
    assert size(30, 4, 2, 5, 64) >= n


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
def test_frequencies(rot):
    """Each scaling against its formula, and what it is for: which pairs slow down, by how much."""
    theta = 10000.0
    inv, ms = tfm.rope_frequencies(theta, rot)
    plain = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    close = lambda a, b: all(math.isclose(x, y, rel_tol=1e-14) for x, y in zip(a, b)) and len(a) == len(b)
    assert inv.dtype == torch.float64 and close(inv.tolist(), plain) and ms == 1.0
    inv, ms = tfm.rope_frequencies(theta, rot, "linear", factor=4.0)
    assert close(inv.tolist(), [f / 4 for f in plain]) and ms == 1.0
    inv, ms = tfm.rope_frequencies(theta, rot, "ntk", factor=8.0)
    if rot > 2:
        assert math.isclose(inv[-1], plain[-1] / 8, rel_tol=1e-12) and inv[0] == 1.0 and ms == 1.0
    turns = [2048 * f / (2 * math.pi) for f in plain]
    inv, ms = tfm.rope_frequencies(theta, rot, "wavelength", factor=8.0, original=2048, low=1.0, high=4.0)
    for i, f in enumerate(inv.tolist()):
        keep = min(max((turns[i] - 1) / 3, 0), 1)
        assert math.isclose(f, plain[i] * (keep + (1 - keep) / 8), rel_tol=1e-13)
    inv, ms = tfm.rope_frequencies(theta, rot, "yarn", factor=16.0, original=2048, low=1.0, high=32.0)
    assert math.isclose(ms, 0.1 * math.log(16) + 1, rel_tol=1e-7)
    ratio = [f / p for f, p in zip(inv.tolist(), plain)]
    assert all(a >= b - 1e-15 for a, b in zip(ratio, ratio[1:]))
    for r, t in zip(ratio, turns):
        if t >= 32:
            assert math.isclose(r, 1, rel_tol=1e-14)
        if rot >= 16 and t * theta ** (2 / rot) < 1:              # more than a pair beyond the one of a single turn
            assert math.isclose(r, 1 / 16, rel_tol=1e-13)
    assert close(tfm.rope_frequencies(theta, rot, "yarn", factor=1.0, original=2048)[0].tolist(), plain)


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(rot=258), dict(theta=1.0), dict(theta=NAN), dict(theta=INF),
                                dict(factor=0.5), dict(factor=NAN), dict(factor=1e7), dict(original=0.0), dict(original=NAN),
                                dict(low=0.0), dict(low=32.0), dict(high=NAN)])
def test_frequencies_refusals(kw):
    d = dict(theta=10000.0, rot=64, scaling="yarn", factor=4.0, original=2048.0, low=1.0, high=32.0)
    d.update(kw)
    with pytest.raises(tfm.TfmError) as e:
        tfm.rope_frequencies(**d)
    assert e.value.status == E


def test_unknown_scaling():
    with pytest.raises(ValueError, match="scaling"):
        tfm.rope_frequencies(10000.0, 64, "cubic")


def test_binding_refuses_host_tensors_and_wrong_layouts():
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)
    cache = (z(2, 2, 40, 32, dtype=torch.int8), z(2, 2, 40, 32, dtype=torch.int8), z(2, 2, 3, dtype=f32), z(2, 2, 3, dtype=f32))
    lens = z(2, dtype=i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tfm.rope_rows(z(3, 2, 32), z(3, 2, 32), z(3, 2, 32), z(3, 2, 32), z(3, dtype=i32), z(16, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        tfm.cache8_write(z(2, 2, 32), z(2, 2, 32), *cache, lens, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tfm.cache8_read(*cache, z(2, 2, 32), z(2, 2, 32), lens, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tfm.cache8_attention(z(2, 4, 32), *cache, z(2, 4, 32), lens, z(64, dtype=torch.uint8), 16)
    with pytest.raises(ValueError, match="both or neither"):
        tfm.rope_rows(z(3, 2, 32), z(3, 2, 32), z(3, 2, 32), None, z(3, dtype=i32), z(16, dtype=torch.float64))
    with pytest.raises(ValueError, match="32 bits"):
        tfm.cache8_attention_workspace_bytes(1 << 32, 4, 2, 1, 64)
