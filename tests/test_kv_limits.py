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


@pytest.mark.parametrize("dim", [64, 96, 128])
def test_the_workspace_is_the_calls(dim):
    """A call of few rows in all asks for an eighth of what many rows do; more tokens, whatever the
    batch, never ask for less."""
    cache = lw.KvCache.empty(3, 2, dim, 16, device="cpu")
    sizes = [lw.lw_kv_workspace_bytes(cache, 8, t, 1) for t in (0, 1, 6, 7, 100, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[2] * 7 < sizes[3]
    assert [lw.lw_kv_workspace_bytes(cache, 8, t, 50) for t in (0, 1, 6, 7, 100, 1 << 20)] == sizes
    # what it cuts off is read by no call: the C call asks for the same
    need = lw.lw_kv_workspace_bytes(lw.KvCache.empty(10, 1, 64, 16, device="cpu"), 1, 3, 2)
    assert c_attention(ws_bytes=need - 1) == lw.LW_ERR_INVALID_ARG


# ---- the binding ------------------------------------------------------------

class OnDevice1(torch.Tensor):
    """A tensor that says it is on cuda:1."""
    device = property(lambda self: torch.device("cuda:1"))

    def get_device(self):
        return 1


def on1(t):
    return t.as_subclass(OnDevice1)


class Calls:
    """Stands in for the library: counts the device calls and does nothing."""

    def __init__(self, real):
        self.real, self.made = real, []

    def __getattr__(self, name):
        if name in ("lw_kv_write", "lw_kv_read", "lw_kv_attention", "lw_kv_workspace_bytes"):
            return lambda *a: self.made.append(name) or 0
        return getattr(self.real, name)


@pytest.fixture
def device1(monkeypatch):
    """A cache that says it is on cuda:1; its calls, by name; and which device is current."""
    cache = lw.KvCache.empty(3, 2, 64, 16, device="cpu")
    cache.index, cache.device = 1, torch.device("cuda:1")
    lib, now = Calls(lw.load()), [1]
    monkeypatch.setattr(lw, "_lib", lib)
    monkeypatch.setattr(lw, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(lw, "_current_device", lambda: now[0], raising=False)
    i32, st = dict(dtype=torch.int32), on1(torch.zeros(1, dtype=torch.int32))
    k, v, slots = on1(torch.zeros(4, 2, 64)), on1(torch.zeros(4, 2, 64)), on1(torch.zeros(4, dtype=torch.int64))
    q, out = on1(torch.zeros(3, 4, 64)), on1(torch.zeros(3, 4, 64))
    start, lens, table = (on1(t) for t in (torch.tensor([0, 1, 3], **i32), torch.zeros(2, **i32),
                                           torch.zeros(2, 5, **i32)))
    ws = on1(torch.zeros(1000, dtype=torch.uint8))
    calls = {"lw_kv_write": lambda k=k, v=v: lw.lw_kv_write(cache, k, v, slots, st),
             "lw_kv_read": lambda k=k, v=v: lw.lw_kv_read(cache, slots, k, v, st),
             "lw_kv_attention": lambda **kw: lw.lw_kv_attention(cache, q, start, lens, table, out, ws, st,
                                                               **{"max_q": 2, **kw}),
             "lw_kv_workspace_bytes": lambda: lw.lw_kv_workspace_bytes(cache, 4, 3, 2)}
    return lib, now, calls


def test_the_current_device_has_to_be_the_caches(device1):
    """The library launches on, and sizes by, the current device: with another one current the calls
    would hand its kernels addresses of the cache's device."""
    lib, now, calls = device1
    for name, call in calls.items():
        call()
        assert lib.made == [name]
        lib.made.clear()
        now[0] = 0
        with pytest.raises(lw.LwError) as e:
            call()
        assert e.value.status == lw.LW_ERR_INVALID_ARG and "current device" in str(e.value)
        assert not lib.made
        now[0] = 1


def test_read_refuses_keys_and_values_in_one_place(device1):
    """Two writers on an element leave either's value: k and v that share memory are refused, rows
    that only lie between one another are not."""
    lib, _, calls = device1
    both = torch.zeros(4, 2, 2, 64)                      # a token's keys, then its values
    flat = torch.zeros(4 * 2 * 64 * 2 + 64)
    fine = [(torch.zeros(4, 2, 64), torch.zeros(4, 2, 64)),
            (both[:, 0], both[:, 1]), (both[:, 1], both[:, 0]),
            (both[:, :, 0], both[:, :, 1]),              # head by head
            (torch.zeros(2, 2, 4, 64)[:, 0].transpose(0, 1), torch.zeros(4, 2, 64)),
            (flat[:512].view(4, 2, 64), flat[512:1024].view(4, 2, 64)),
            # different strides in one buffer: k's tokens before v's heads
            (flat[:512].view(4, 2, 64), flat[512:1024].view(2, 4, 64).transpose(0, 1))]
    for k, v in fine:
        calls["lw_kv_read"](on1(k), on1(v))
        assert lib.made == ["lw_kv_read"]
        lib.made.clear()
    k = torch.zeros(4, 2, 64)
    wrong = [(k, k), (k, k.view(2, 4, 64).transpose(0, 1)),
             (flat[:512].view(4, 2, 64), flat[448:960].view(4, 2, 64)),          # the last head
             (flat[:512].view(4, 2, 64), flat[511:1023].view(4, 2, 64)),         # one element
             (both[:, 0], both.view(-1)[64:64 + 960].as_strided((4, 2, 64), (256, 64, 1)))]
    for k, v in wrong:
        with pytest.raises(lw.LwError) as e:
            calls["lw_kv_read"](on1(k), on1(v))
        assert e.value.status == lw.LW_ERR_INVALID_ARG and "overlap" in str(e.value)
        assert not lib.made
        calls["lw_kv_write"](on1(k), on1(v))             # (rows that are read may)
        lib.made.clear()
