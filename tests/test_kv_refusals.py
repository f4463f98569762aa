"""What the 4-bit key/value cache's calls refuse, on the CPU: the binding's
checks of tensors (the library handle is swapped for a guard that fails the
test if a device call is reached), and the C calls' own checks of shapes,
types, strides, addresses and sizes (made-up addresses; every case is refused
before a launch)."""
import ctypes

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
FAKE = 0x7F0000000000
KEEP = lw.load


class _Guard:
    """Stands in for the loaded library: its device calls are failures."""

    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        if name in ("lw_kv_write", "lw_kv_read", "lw_kv_attention"):
            raise AssertionError(f"{name} was called although the binding should have refused")
        return getattr(self._real, name)


@pytest.fixture
def guarded(monkeypatch):
    monkeypatch.setattr(lw, "_lib", _Guard(lw.load()))


def cache(heads=2, dim=64, page=16, pages=3):
    return lw.KvCache.empty(pages, heads, dim, page, device="cpu")


def refused(call, *words):
    with pytest.raises(lw.LwError) as e:
        call()
    assert e.value.status == lw.LW_ERR_INVALID_ARG
    for w in words:
        assert w in str(e.value), str(e.value)


def test_sizes():
    assert [lw.lw_kv_tile_bytes(d) for d in (64, 96, 128)] == [1280, 1952, 2560]
    assert [lw.lw_kv_tile_bytes(d) for d in (0, 32, 80, 127, 256, -64)] == [0] * 6
    assert lw.lw_kv_page_bytes(8, 128, 64) == 8 * 4 * 2560
    for heads, dim, page in ((0, 64, 16), (-1, 64, 16), (1, 64, 0), (1, 64, 17), (1, 64, -16), (1, 72, 16)):
        assert lw.lw_kv_page_bytes(heads, dim, page) == 0
    c = cache()
    assert c.n_pages == 3 and lw.lw_kv_workspace_bytes(c, 4, 10, 2) > 0
    for heads, tokens, batch in ((3, 10, 2), (0, 10, 2), (4, -1, 2), (4, 10, 0)):
        assert lw.lw_kv_workspace_bytes(c, heads, tokens, batch) == 0


def test_cache_views():
    size = lw.lw_kv_page_bytes(2, 64, 16)
    refused(lambda: lw.KvCache(torch.zeros(size + 1, dtype=torch.uint8), 2, 64, 16), "multiple")
    refused(lambda: lw.KvCache(torch.zeros(size - 1, dtype=torch.uint8), 2, 64, 16), "pages", "needs")
    refused(lambda: lw.KvCache(torch.zeros(size, dtype=torch.uint8), 2, 80, 16), "head_dim")
    refused(lambda: lw.KvCache(torch.zeros(size, dtype=torch.uint8), 2, 64, 24), "page_tokens")
    refused(lambda: lw.KvCache(torch.zeros(size, 2, dtype=torch.uint8)[:, 0], 2, 64, 16), "contiguous")
    refused(lambda: lw.KvCache(None, 2, 64, 16), "pages")


def rows(n=4, heads=2, dim=64, dtype=torch.float32):
    return torch.zeros(n, heads, dim, dtype=dtype)


@pytest.mark.parametrize("write", [True, False])
def test_rows(guarded, write):
    c, st, slots = cache(), torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)

    def call(k=None, v=None, s=slots, d=st):
        k = rows() if k is None else k
        v = rows() if v is None else v
        if write:
            lw.lw_kv_write(c, k, v, s, d)
        else:
            lw.lw_kv_read(c, s, k, v, d)

    refused(lambda: call(), "pages on cpu")                    # everything right but the device
    refused(lambda: call(k=rows(dtype=torch.float64)), "k", "float64")
    refused(lambda: call(v=rows(dtype=torch.bfloat16)), "v", "bfloat16")
    refused(lambda: call(k=rows(3)), "k", "shape")
    refused(lambda: call(v=rows(heads=1)), "v", "shape")
    refused(lambda: call(k=rows(dim=96)), "k", "shape")
    refused(lambda: call(k=torch.zeros(4, 128)), "k", "shape")
    refused(lambda: call(k=torch.zeros(4, 64, 2).transpose(1, 2)), "k", "strided")
    refused(lambda: call(k=[1.0]), "k", "Tensor")
    refused(lambda: call(s=slots.int()), "slots", "int32")
    refused(lambda: call(s=torch.zeros(8, dtype=torch.int64)[::2]), "slots", "contiguous")
    refused(lambda: call(s=torch.zeros(2, 2, dtype=torch.int64)), "slots")
    refused(lambda: call(s=None), "slots", "Tensor")
    refused(lambda: call(d=torch.zeros(1)), "d_status")
    refused(lambda: call(d=torch.zeros(0, dtype=torch.int32)), "d_status")
    if not write:   # rows that share elements may be read from, not written to
        refused(lambda: call(k=torch.zeros(1, 2, 64).expand(4, 2, 64)), "k", "overlap")
        refused(lambda: call(v=torch.zeros(4, 1, 64).expand(4, 2, 64)), "v", "overlap")


def test_attention(guarded):
    c = cache()
    i32 = dict(dtype=torch.int32)
    good = dict(q=rows(3, 4), q_start=torch.tensor([0, 1, 3], **i32), kv_len=torch.zeros(2, **i32),
                page_table=torch.zeros(2, 5, **i32), out=rows(3, 4), ws=torch.zeros(1000, dtype=torch.uint8),
                d_status=torch.zeros(1, **i32))

    def call(**kw):
        a = {**good, **kw}
        lw.lw_kv_attention(c, a.pop("q"), a.pop("q_start"), a.pop("kv_len"), a.pop("page_table"), a.pop("out"),
                           a.pop("ws"), a.pop("d_status"), max_q=a.pop("max_q", 2), **a)

    refused(lambda: call(), "pages on cpu")
    refused(lambda: call(q=rows(3, 3)), "q", "multiple of 2")
    refused(lambda: call(q=rows(3, 4, 96)), "q", "shape")
    refused(lambda: call(q=torch.zeros(3, 256)), "q", "shape")
    refused(lambda: call(q=rows(3, 4, dtype=torch.float64)), "q", "float64")
    refused(lambda: call(q=None), "q", "Tensor")
    refused(lambda: call(q=torch.zeros(3, 64, 4).transpose(1, 2)), "q", "strided")
    refused(lambda: call(out=rows(3, 4, dtype=torch.bfloat16)), "out", "bfloat16")
    refused(lambda: call(out=rows(2, 4)), "out", "shape")
    refused(lambda: call(out=torch.zeros(1, 4, 64).expand(3, 4, 64)), "out", "overlap")
    refused(lambda: call(q_start=torch.zeros(2, **i32)), "q_start", "3")
    refused(lambda: call(q_start=torch.zeros(3)), "q_start", "float32")
    refused(lambda: call(kv_len=torch.zeros(2, dtype=torch.int64)), "kv_len", "int64")
    refused(lambda: call(page_table=torch.zeros(3, 5, **i32)), "page_table")
    refused(lambda: call(page_table=torch.zeros(2, 5)), "page_table")
    refused(lambda: call(page_table=torch.zeros(5, 2, **i32).t()), "page_table", "contiguous")
    refused(lambda: call(ws=torch.zeros(4, 4)[:, 0]), "ws")
    refused(lambda: call(lse=torch.zeros(3, 4, dtype=torch.float64)), "lse")
    refused(lambda: call(lse=torch.zeros(11)), "lse")
    refused(lambda: call(d_status=None), "d_status")
    refused(lambda: call(max_q=1.5), "max_q")


# ---- the C calls ------------------------------------------------------------

def view(**kw):
    v = lw.LwKvCache(FAKE, 10, 2, 64, 16, 0)
    for k, x in kw.items():
        setattr(v, k, x)
    return v


def status(fn, *args):
    lib = lw.load()
    st = getattr(lib, fn)(*args)
    return st, lib.lw_last_error().decode()


BAD_CACHES = [(dict(pages=None), lw.LW_ERR_INVALID_ARG), (dict(pages=FAKE + 8), lw.LW_ERR_INVALID_ARG),
              (dict(n_pages=0), lw.LW_ERR_SHAPE), (dict(n_pages=1 << 40), lw.LW_ERR_SHAPE),
              (dict(kv_heads=0), lw.LW_ERR_SHAPE), (dict(page_tokens=8), lw.LW_ERR_SHAPE),
              (dict(head_dim=80), lw.LW_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("fn", ["lw_kv_write", "lw_kv_read"])
def test_c_rows(fn):
    def call(v=None, k=(FAKE, 128, 64, 0, 0), w=(FAKE, 128, 64, 0, 0), slots=FAKE, n=4):
        c = ctypes.byref(view() if v is None else v)
        k = None if k is None else lw._KV_ROWS.pack(*k)
        w = None if w is None else lw._KV_ROWS.pack(*w)
        args = (c, k, w, slots, n) if fn == "lw_kv_write" else (c, slots, n, k, w)
        return status(fn, *args, None, None)

    for kw, want in BAD_CACHES:
        st, msg = call(view(**kw))
        assert st == want and msg, kw
    for kw, want in [(dict(k=None), lw.LW_ERR_INVALID_ARG), (dict(w=(0, 128, 64, 0, 0)), lw.LW_ERR_INVALID_ARG),
                     (dict(k=(FAKE + 2, 128, 64, 0, 0)), lw.LW_ERR_INVALID_ARG),
                     (dict(k=(FAKE, 128, 64, 7, 0)), lw.LW_ERR_UNSUPPORTED),
                     (dict(k=(FAKE, 128, 64, 1, 0)), lw.LW_ERR_INVALID_ARG),     # keys fp16, values fp32
                     (dict(slots=0), lw.LW_ERR_INVALID_ARG), (dict(slots=FAKE + 4), lw.LW_ERR_INVALID_ARG),
                     (dict(n=-1), lw.LW_ERR_INVALID_ARG), (dict(n=1 << 40), lw.LW_ERR_SHAPE)]:
        st, msg = call(**kw)
        assert st == want and msg, kw
    st, _ = status(fn, None, *((None, None, None, 0) if fn == "lw_kv_write" else (None, 0, None, None)), None, None)
    assert st == lw.LW_ERR_INVALID_ARG
    assert call(n=0)[0] == lw.LW_OK   # nothing to do, nothing launched


def test_c_attention():
    fields = ["q", "qt", "qh", "out", "ot", "oh", "lse", "q_start", "kv_len", "page_table", "table_stride", "q_tokens",
              "table_width", "dtype", "batch", "q_heads", "max_q", "causal", "window", "scale"]
    good = dict(q=FAKE, qt=256, qh=64, out=FAKE, ot=256, oh=64, lse=0, q_start=FAKE, kv_len=FAKE, page_table=FAKE,
                table_stride=5, q_tokens=3, table_width=5, dtype=0, batch=2, q_heads=4, max_q=2, causal=1, window=0,
                scale=0.125)
    need = lw.load().lw_kv_workspace_bytes(ctypes.byref(view()), 4, 3, 2)

    def call(v=None, ws=FAKE, ws_bytes=need, **kw):
        a = {**good, **kw}
        return status("lw_kv_attention", ctypes.byref(view() if v is None else v),
                      lw._KV_ATTN.pack(*(a[f] for f in fields)), ws, ws_bytes, None, None)

    for kw, want in BAD_CACHES:
        st, msg = call(view(**kw))
        assert st == want and msg, kw
    inv, shp, uns = lw.LW_ERR_INVALID_ARG, lw.LW_ERR_SHAPE, lw.LW_ERR_UNSUPPORTED
    for kw, want in [(dict(q=0), inv), (dict(out=0), inv), (dict(q_start=0), inv), (dict(kv_len=0), inv),
                     (dict(page_table=0), inv), (dict(q=FAKE + 2), inv), (dict(lse=FAKE + 1), inv),
                     (dict(q_start=FAKE + 2), inv), (dict(dtype=3), uns), (dict(batch=0), shp),
                     (dict(batch=70000), shp), (dict(q_heads=3), shp), (dict(q_heads=0), shp),
                     (dict(q_tokens=-1), shp), (dict(q_tokens=1 << 33), shp), (dict(max_q=-1), inv),
                     (dict(causal=2), inv), (dict(window=-1), inv), (dict(scale=float("nan")), inv),
                     (dict(scale=float("inf")), inv), (dict(table_width=-1), shp),
                     (dict(table_width=1 << 30), shp), (dict(table_stride=-1), shp),
                     (dict(ws=0), inv), (dict(ws=FAKE + 8), inv), (dict(ws_bytes=need - 1), inv)]:
        st, msg = call(**kw)
        assert st == want and msg, (kw, st, msg)
    assert status("lw_kv_attention", ctypes.byref(view()), None, FAKE, need, None, None)[0] == inv
    assert call(q_tokens=0)[0] == lw.LW_OK   # no queries: nothing launched
