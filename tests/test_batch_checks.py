"""Host-side checks of the batched-serving entry points (packed prompts, a shared
prefix, drafted tokens): every limit the header states is refused before any
pointer is read, empty calls return at once, workspace sizes, and the binding's
refusals.  No GPU is touched; the pointers are aligned but point nowhere."""
import ctypes

import pytest
import torch

from decoder_only_transformer_gb300 import tfm

B16, F32 = tfm.TFM_BF16, tfm.TFM_FP32
E, U, OK = tfm.TFM_EINVAL, tfm.TFM_EUNSUPPORTED, tfm.TFM_OK
A = ctypes.c_void_p(256)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return tfm.load()


def _packed(lib, **kw):
    d = dict(q=A, k=A, v=A, o=A, cu=A, n_seq=3, T=100, H=4, Hkv=2, dh=64, strides=None, scale=0.0,
             window=0, mode=B16, ws=A, nbytes=1 << 20)
    d.update(kw)
    st = d["strides"]
    if st is not None:
        d["strides"] = (ctypes.c_int64 * 8)(*st)
    return lib.tfm_packed_attention(*(d[k] for k in ("q", "k", "v", "o", "cu", "n_seq", "T", "H", "Hkv", "dh",
                                                     "strides", "scale", "window", "mode", "ws", "nbytes")), None)


def _prefix(lib, **kw):
    d = dict(q=A, kp=A, vp=A, kc=A, vc=A, o=A, lens=A, B=3, H=4, Hkv=2, T=2, P=10, maxp=16, maxs=32, dh=64,
             scale=0.0, ws=A, nbytes=1 << 30)
    d.update(kw)
    return lib.tfm_prefix_attention(*(d[k] for k in ("q", "kp", "vp", "kc", "vc", "o", "lens", "B", "H", "Hkv", "T",
                                                     "P", "maxp", "maxs", "dh", "scale", "ws", "nbytes")), None)


def _verify(lib, **kw):
    d = dict(target=A, ldt=104, dl=A, ldd=104, draft=A, nd=A, u=A, noise=A, ldn=104, B=3, K=4, V=101, temp=1.0,
             tokens=A, acc=A, ws=A, nbytes=1 << 20)
    d.update(kw)
    return lib.tfm_verify_draft(*(d[k] for k in ("target", "ldt", "dl", "ldd", "draft", "nd", "u", "noise", "ldn",
                                                 "B", "K", "V", "temp", "tokens", "acc", "ws", "nbytes")), None)


DENSE = [256, 64, 128, 64, 128, 64, 256, 64]


def _stride(i, v):
    s = list(DENSE)
    s[i] = v
    return s


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), E), (dict(T=(1 << 30) + 1), E), (dict(n_seq=-1), E), (dict(n_seq=(1 << 20) + 1), E),
    (dict(H=0), E), (dict(Hkv=0), E), (dict(Hkv=3), E), (dict(dh=0), E), (dict(mode=7), E),
    (dict(window=-1), E), (dict(scale=NAN), E), (dict(scale=INF), E),
    (dict(T=1 << 30, H=512, Hkv=512), E),                    # items beyond int32
    (dict(dh=48), U), (dict(dh=256), U), (dict(dh=6, mode=F32), U), (dict(dh=132, mode=F32), U),
    (dict(q=None), E), (dict(k=None), E), (dict(v=None), E), (dict(o=None), E), (dict(cu=None), E), (dict(ws=None), E),
    (dict(q=ctypes.c_void_p(264)), E), (dict(o=ctypes.c_void_p(258)), E), (dict(ws=ctypes.c_void_p(260)), E),
    (dict(cu=ctypes.c_void_p(258)), E),
    (dict(strides=_stride(0, 63)), E), (dict(strides=_stride(1, 0)), E), (dict(strides=_stride(3, -64)), E),
    (dict(strides=_stride(4, 132)), E),                      # 264 bytes: not a multiple of 16
    (dict(strides=_stride(6, 1 << 39)), E),
    (dict(nbytes=0), E),
    (dict(T=0), OK), (dict(n_seq=0), OK), (dict(T=0, q=None, k=None, v=None, o=None, cu=None, ws=None), OK),
    (dict(T=0, dh=48), U), (dict(n_seq=0, Hkv=3), E),       # the other arguments are still checked
    (dict(T=1, n_seq=0, strides=_stride(0, 1)), OK),         # the stride of a single row is never used
])
def test_packed_attention_refusals(lib, kw, status):
    assert _packed(lib, **kw) == status, lib.tfm_last_error()
    if status != OK:
        assert lib.tfm_last_error()


def test_packed_attention_workspace(lib):
    n = lib.tfm_packed_attention_workspace_bytes(1000, 7)
    assert n > 0 and _packed(lib, T=1000, n_seq=7, nbytes=n - 1) == E
    assert b"workspace too small" in lib.tfm_last_error()
    assert lib.tfm_packed_attention_workspace_bytes(-1, 7) == 0
    assert lib.tfm_packed_attention_workspace_bytes(10, -1) == 0
    assert lib.tfm_packed_attention_workspace_bytes((1 << 30) + 1, 1) == 0
    assert lib.tfm_packed_attention_workspace_bytes(4000, 7) >= n
    assert lib.tfm_packed_attention_workspace_bytes(1000, 70) >= n


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), E), (dict(B=4097), E), (dict(H=0), E), (dict(Hkv=0), E), (dict(Hkv=3), E), (dict(T=0), E),
    (dict(B=4096, H=4096, Hkv=4096, T=2), E),
    (dict(P=-1), E), (dict(P=17), E), (dict(maxs=0), E), (dict(maxs=1 << 30), E),
    (dict(Hkv=2, H=2, P=1, maxp=1 << 30), E),
    (dict(scale=NAN), E), (dict(dh=48), U), (dict(dh=256), U), (dict(T=65), U),
    (dict(q=None), E), (dict(kc=None), E), (dict(vc=None), E), (dict(o=None), E), (dict(lens=None), E),
    (dict(ws=None), E), (dict(kp=None), E), (dict(vp=None), E),
    (dict(kp=ctypes.c_void_p(264)), E), (dict(o=ctypes.c_void_p(264)), E), (dict(lens=ctypes.c_void_p(257)), E),
    (dict(nbytes=0), E),
    (dict(B=0), OK), (dict(B=0, q=None, kc=None, o=None, lens=None, ws=None), OK), (dict(B=0, T=0), E),
])
def test_prefix_attention_refusals(lib, kw, status):
    assert _prefix(lib, **kw) == status, lib.tfm_last_error()
    if status != OK:
        assert lib.tfm_last_error()


def test_prefix_attention_workspace(lib):
    n = lib.tfm_prefix_attention_workspace_bytes(3, 4, 2, 2, 64)
    assert n > 0 and _prefix(lib, nbytes=n - 1) == E
    assert lib.tfm_prefix_attention_workspace_bytes(-1, 4, 2, 2, 64) == 0
    assert lib.tfm_prefix_attention_workspace_bytes(3, 4, 3, 2, 64) == 0
    assert lib.tfm_prefix_attention_workspace_bytes(3, 4, 2, 2, 48) == 0
    assert lib.tfm_prefix_attention_workspace_bytes(3, 4, 2, 65, 64) == 0
    assert lib.tfm_prefix_attention_workspace_bytes(30, 4, 2, 2, 64) >= n


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), E), (dict(K=-1), E), (dict(K=65), E), (dict(V=0), E), (dict(V=(1 << 30) + 1), E),
    (dict(B=1 << 20, K=1), E), (dict(temp=-0.5), E), (dict(temp=NAN), E), (dict(temp=INF), E),
    (dict(ldt=100), E), (dict(ldt=102), E), (dict(ldd=100), E), (dict(ldn=103), E),
    (dict(target=None), E), (dict(dl=None), E), (dict(draft=None), E), (dict(u=None), E), (dict(noise=None), E),
    (dict(tokens=None), E), (dict(acc=None), E), (dict(ws=None), E),
    (dict(target=ctypes.c_void_p(264)), E), (dict(noise=ctypes.c_void_p(264)), E), (dict(dl=ctypes.c_void_p(264)), E),
    (dict(draft=ctypes.c_void_p(258)), E), (dict(nd=ctypes.c_void_p(258)), E), (dict(u=ctypes.c_void_p(258)), E),
    (dict(tokens=ctypes.c_void_p(258)), E), (dict(acc=ctypes.c_void_p(258)), E),
    (dict(nbytes=0), E),
    (dict(temp=0.0, target=None), E), (dict(temp=0.0, draft=None), E),
    (dict(B=0), OK), (dict(B=0, target=None, draft=None, tokens=None, ws=None), OK), (dict(B=0, V=0), E),
])
def test_verify_draft_refusals(lib, kw, status):
    assert _verify(lib, **kw) == status, lib.tfm_last_error()
    if status != OK:
        assert lib.tfm_last_error()


def test_verify_draft_workspace(lib):
    n = lib.tfm_verify_draft_workspace_bytes(3, 4, 101)
    assert n > 0 and _verify(lib, nbytes=n - 1) == E
    assert lib.tfm_verify_draft_workspace_bytes(-1, 4, 101) == 0
    assert lib.tfm_verify_draft_workspace_bytes(3, 65, 101) == 0
    assert lib.tfm_verify_draft_workspace_bytes(3, 4, 0) == 0
    assert lib.tfm_verify_draft_workspace_bytes(30, 4, 50257) > n


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors_and_wrong_layouts():
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    ws = _cpu(64, dtype=u8)
    calls = [
        lambda: tfm.packed_attention(_cpu(8, 2, 32), _cpu(8, 2, 32), _cpu(8, 2, 32), _cpu(8, 2, 32),
                                     _cpu(2, dtype=i32), ws),
        lambda: tfm.prefix_attention(_cpu(1, 2, 1, 32), _cpu(2, 4, 32), _cpu(2, 4, 32), _cpu(1, 2, 4, 32),
                                     _cpu(1, 2, 4, 32), _cpu(1, 1, 64), _cpu(1, dtype=i32), ws),
        lambda: tfm.verify_draft(_cpu(3, 8, dtype=f32), _cpu(2, 8, dtype=f32), _cpu(1, 2, dtype=i32), None,
                                 _cpu(1, 2, dtype=f32), _cpu(1, 8, dtype=f32), 8, _cpu(1, 3, dtype=i32),
                                 _cpu(1, dtype=i32), ws),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("call,kw,status", [
    (_verify, dict(temp=1e-31), E), (_verify, dict(temp=1e31), E),
    (_verify, dict(V=(1 << 24) + 1, ldt=1 << 25, ldd=1 << 25, ldn=1 << 25), E),
    (_packed, dict(T=1, n_seq=1, H=(1 << 30) + 2, strides=None), E),      # items beyond int32 less a grid
    (_packed, dict(T=0, n_seq=1 << 20, H=1024, Hkv=1024, strides=None), OK),
    (_packed, dict(T=0, n_seq=1 << 20, H=1026, Hkv=2, strides=None), E),
])
def test_limits_of_the_arithmetic(lib, call, kw, status):
    assert call(lib, **kw) == status, lib.tfm_last_error()
