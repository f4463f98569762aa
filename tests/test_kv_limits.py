"""The ends of the ranges that the 4-bit cache's calls take, on the CPU: sizes
at their 32-bit limits, and what the binding refuses of devices, overlapping
rows and numbers.  Nothing here reaches a launch."""
import ctypes

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
FAKE = 0x7F0000000000


def c_attention(kv_heads=1, page_tokens=16, ws_bytes=0, **kw):
    """The C call on made-up addresses; ws_bytes = 0 is refused last, so that no case launches."""
    a = dict(q=FAKE, qt=0, qh=64, out=FAKE, ot=256, oh=64, lse=0, q_start=FAKE, kv_len=FAKE, page_table=FAKE,
             table_stride=5, q_tokens=3, table_width=5, dtype=0, batch=2, q_heads=1, max_q=2, causal=1, window=0,
             scale=0.125)
    a.update(kw)
    view = lw.LwKvCache(FAKE, 10, kv_heads, 64, page_tokens, 0)
    lib = lw.load()
    return lib.lw_kv_attention(ctypes.byref(view), lw._KV_ATTN.pack(*a.values()), FAKE, ws_bytes, None, None)


@pytest.mark.parametrize("kw", [dict(q_tokens=2 ** 31 - 1), dict(q_tokens=2 ** 31 - 255), dict(max_q=2 ** 31 - 255),
                                dict(q_tokens=(2 ** 31 - 512) // 8, q_heads=8),
                                dict(table_width=2 ** 27 - 1)])
def test_rows_and_keys_stay_within_32_bits(kw):
    """A row tile may run 255 rows past the last row, a unit 256 keys past the last key: sizes where
    such a number would not fit 31 bits are refused."""
    assert c_attention(**kw) == lw.LW_ERR_SHAPE


def test_the_largest_sizes_are_taken():
    """Up to the limit the sizes pass (the missing workspace is what is refused then)."""
    for kw in (dict(q_tokens=2 ** 31 - 1024), dict(max_q=2 ** 31 - 1024), dict(table_width=2 ** 27 - 64)):
        assert c_attention(**kw) == lw.LW_ERR_INVALID_ARG
        assert b"workspace" in lw.load().lw_last_error()
