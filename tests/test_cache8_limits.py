"""The ends of the 8-bit cache's ranges, on the host.  Every call is refused (a pointer is missing, if nothing else is
wrong), so that none launches anything, with or without a GPU; the message says which check it was."""
import ctypes

import pytest

from decoder_only_transformer_gb300 import tfm

A = ctypes.c_void_p(256)
E = tfm.TFM_EINVAL


def _message(status):
    assert status == E
    return tfm.load().tfm_last_error().decode()


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("dh", [32, 128])
@pytest.mark.parametrize("call", ["write", "read", "attention"])
def test_positions_that_ints_hold(call, dh, block):
    """The end of the last position's block (p0 + block) and of its tile (key + 64, and the rounding of a length to
    tiles) are ints in the kernels: above 2^31 - 128 a write would take rows behind the last new one, and attention would
    see one tile."""
    lib = tfm.load()

    def message(max_seq):
        if call == "attention":
            return _message(lib.tfm_cache8_attention(None, A, A, A, A, A, A, A, 1, 1, 1, 1, 1, dh, max_seq, block, None, 0, 0,
                                                     0.0, A, 1 << 30, None))
        rows, cache = (None, A), (A, A, A, A)
        f, args = (lib.tfm_cache8_write, rows + cache) if call == "write" else (lib.tfm_cache8_read, cache + rows)
        return _message(f(*args, A, A, 1, 1, 1, dh, max_seq, block, None, 0, tfm.TFM_BF16, None))

    last = 2 ** 31 - 256
    for n in (last, last - 1, 2 ** 30):
        assert "NULL pointer" in message(n)
        # what the kernels compute from it stays below 2^31: the end of a block, of a warp's step, of a rounded length
        assert (n - 1) // block * block + block < 2 ** 31 and n + 64 + 48 + 16 < 2 ** 31
    for n in (last + 1, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 63, 2 ** 31 - 1, 0, -1):
        assert "max_seq" in message(n)


def test_strides_of_no_heads_are_not_read():
    """With Hkv = 0 neither k nor its strides are used, whatever they hold."""
    lib = tfm.load()

    def message(Hkv, kt, kh):
        strides = (ctypes.c_int64 * 8)(256, 64, kt, kh, 256, 64, kt, kh)
        return _message(lib.tfm_rope_rows(None, None, A, None, A, A, 10, 4, Hkv, 64, 64, 1, strides, 1.0, tfm.TFM_BF16, None))

    for kt, kh in ((0, 0), (-1, 7), (1 << 40, 1 << 40), (128, 64)):
        assert "NULL pointer" in message(0, kt, kh)
    assert "k token stride" in message(2, 0, 64) and "k head stride" in message(2, 128, 0)
    assert "NULL pointer" in message(1, 64, 0)               # the head stride of one head is not read either
