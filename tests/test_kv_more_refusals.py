"""What the calls around the 4-bit cache refuse -- rotary write, accumulated weight, eviction, block-sparse attention
-- on the CPU: the binding's checks of tensors (the library handle is swapped for a guard that fails the test if a
device call is reached), and the C calls' own checks (made-up addresses; every case is refused before a launch)."""
import ctypes

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
FAKE = 0x7F0000000000
CALLS = ("lw_rotary_table", "lw_kv_write_rotary", "lw_kv_weigh", "lw_kv_evict", "lw_kv_summarise",
         "lw_kv_attention_blocks")
INV, SHP, UNS = lw.LW_ERR_INVALID_ARG, lw.LW_ERR_SHAPE, lw.LW_ERR_UNSUPPORTED
I32, I64 = dict(dtype=torch.int32), dict(dtype=torch.int64)


class _Guard:
    """Stands in for the loaded library: its device calls are failures."""

    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        if name in CALLS:
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
    assert e.value.status == INV
    for w in words:
        assert w in str(e.value), str(e.value)


def rows(n=4, heads=2, dim=64, dtype=torch.float32):
    return torch.zeros(n, heads, dim, dtype=dtype)


def st():
    return torch.zeros(1, **I32)


# ---- the binding --------------------------------------------------------------

def test_table(guarded):
    refused(lambda: lw.lw_rotary_table(torch.zeros(4, 8)), "table", "cpu")
    refused(lambda: lw.lw_rotary_table(torch.zeros(4, 8, dtype=torch.float64)), "table", "float32")
    refused(lambda: lw.lw_rotary_table(torch.zeros(4, 8).t()), "table", "contiguous")
    refused(lambda: lw.lw_rotary_table(torch.zeros(8)), "table")
    refused(lambda: lw.lw_rotary_table(None), "table")


def test_rotary(guarded):
    c = cache()
    good = dict(k=rows(), v=rows(), slots=torch.zeros(4, **I64), positions=torch.zeros(4, **I64),
                table=torch.zeros(10, 64), d_status=st(), q=rows(heads=6), q_out=rows(heads=6))

    def call(**kw):
        a = {**good, **kw}
        lw.lw_kv_write_rotary(c, a.pop("k"), a.pop("v"), a.pop("slots"), a.pop("positions"), a.pop("table"),
                              a.pop("d_status"), **a)

    refused(lambda: call(), "pages on cpu")                     # everything right but the device
    refused(lambda: call(q=None, q_out=None), "pages on cpu")
    buf = rows(4, 10)
    packed = dict(q=buf[:, :6], q_out=buf[:, :6], k=buf[:, 6:8], v=buf[:, 8:])
    refused(lambda: call(**packed), "pages on cpu")
    refused(lambda: call(k=rows(3)), "k", "shape")
    refused(lambda: call(v=rows(dtype=torch.float16)), "v", "float16")
    refused(lambda: call(v=rows(dtype=torch.int32)), "v", "int32")
    refused(lambda: call(slots=torch.zeros(4, **I32)), "slots", "int32")
    refused(lambda: call(slots=torch.zeros(5, **I64)), "positions", "5")
    refused(lambda: call(positions=torch.zeros(4)), "positions", "float32")
    refused(lambda: call(positions=torch.zeros(8, **I64)[::2]), "positions", "contiguous")
    refused(lambda: call(positions=None), "positions", "Tensor")
    refused(lambda: call(table=torch.zeros(10, 64, dtype=torch.float64)), "table")
    refused(lambda: call(table=torch.zeros(10, 128)[:, :64]), "table", "contiguous")
    refused(lambda: call(table=torch.zeros(640)), "table")
    refused(lambda: call(q=None), "together")
    refused(lambda: call(q_out=None), "together")
    refused(lambda: call(q=rows(heads=6, dtype=torch.float16)), "q")
    refused(lambda: call(q_out=rows(heads=5)), "q_out", "shape")
    refused(lambda: call(q=rows(5, 6)), "q", "shape")
    refused(lambda: call(q_out=torch.zeros(1, 6, 64).expand(4, 6, 64)), "q_out", "overlap")
    refused(lambda: call(d_status=torch.zeros(1)), "d_status")
    wide = torch.zeros(5, 6, 64)
    refused(lambda: call(q=wide[:4], q_out=wide[1:]), "q_out", "overlap")     # a token on
    refused(lambda: call(q_out=buf[:, :6], k=buf[:, 5:7]), "q_out", "k")      # a head of both
    refused(lambda: call(q=buf[:, 2:8], q_out=buf[:, 2:8], v=buf[:, 6:8]), "q_out", "v")
    one = torch.zeros(4 * 6 * 64 + 2 * 64)
    refused(lambda: call(q_out=one[:-128].view(4, 6, 64), k=one[-4 * 128:].view(4, 2, 64)), "q_out", "k")
    refused(lambda: call(q_out=rows(4, 6).view(4, 6, 64), k=rows(4, 2, 96)), "k", "shape")


def test_weigh(guarded):
    c = cache()
    good = dict(q=rows(3, 4), lse=torch.zeros(3, 4), q_start=torch.tensor([0, 1, 3], **I32),
                kv_len=torch.zeros(2, **I32), page_table=torch.zeros(2, 5, **I32), weights=torch.zeros(2, 2, 80),
                ws=torch.zeros(16, dtype=torch.uint8), d_status=st())

    def call(**kw):
        a = {**good, **kw}
        lw.lw_kv_weigh(c, a.pop("q"), a.pop("lse"), a.pop("q_start"), a.pop("kv_len"), a.pop("page_table"),
                       a.pop("weights"), a.pop("ws"), a.pop("d_status"), max_q=a.pop("max_q", 2), **a)

    refused(lambda: call(), "pages on cpu")
    refused(lambda: call(add_to=good["weights"]), "pages on cpu")
    refused(lambda: call(add_to=torch.zeros(2, 1, 80).expand(2, 2, 80)), "pages on cpu")   # read, not written
    refused(lambda: call(q=rows(3, 3)), "q", "multiple of 2")
    refused(lambda: call(q=rows(3, 4, 96)), "q", "shape")
    refused(lambda: call(lse=torch.zeros(11)), "lse")
    refused(lambda: call(lse=torch.zeros(3, 4, dtype=torch.float64)), "lse")
    refused(lambda: call(q_start=torch.zeros(2, **I32)), "q_start", "3")
    refused(lambda: call(kv_len=torch.zeros(2, **I64)), "kv_len", "int64")
    refused(lambda: call(page_table=torch.zeros(3, 5, **I32)), "page_table")
    refused(lambda: call(weights=torch.zeros(2, 3, 80)), "weights", "shape")
    refused(lambda: call(weights=torch.zeros(2, 2, 80, dtype=torch.float16)), "weights", "float32")
    refused(lambda: call(weights=torch.zeros(2, 80, 2).transpose(1, 2)), "weights", "strided")
    refused(lambda: call(weights=torch.zeros(2, 1, 80).expand(2, 2, 80)), "weights", "overlap")
    refused(lambda: call(add_to=torch.zeros(2, 2, 79)), "add_to", "shape")
    whole = torch.zeros(2, 2, 81)
    refused(lambda: call(weights=whole[..., 1:], add_to=whole[..., :80]), "add_to", "overlaps")
    refused(lambda: call(ws=torch.zeros(4, 4)[:, 0]), "ws")
    refused(lambda: call(d_status=None), "d_status")
    refused(lambda: call(max_q=1.5), "max_q")


def test_evict(guarded):
    c = cache()
    good = dict(weights=torch.zeros(2, 2, 80), kv_len=torch.zeros(2, **I32), page_table=torch.zeros(2, 5, **I32),
                out_table=torch.zeros(2, 2, **I32), out_len=torch.zeros(2, **I32), out_weights=torch.zeros(2, 2, 20),
                kept=torch.zeros(2, 2, 20, **I32), d_status=st())

    def call(**kw):
        a = {**good, **kw}
        lw.lw_kv_evict(c, a.pop("weights"), a.pop("kv_len"), a.pop("page_table"), a.pop("out_table"), a.pop("out_len"),
                       a.pop("out_weights"), a.pop("kept"), a.pop("d_status"), keep=a.pop("keep", 20), **a)

    refused(lambda: call(), "pages on cpu")
    refused(lambda: call(out_weights=None), "pages on cpu")
    refused(lambda: call(out_weights=good["weights"]), "pages on cpu")
    refused(lambda: call(keep=2.5), "keep")
    refused(lambda: call(first="1"), "first")
    refused(lambda: call(kept=torch.zeros(2, 2, 19, **I32)), "kept")
    refused(lambda: call(kept=torch.zeros(2, 2, 20, **I64)), "kept")
    refused(lambda: call(kept=torch.zeros(2, 2, 40, **I32)[..., ::2]), "kept", "contiguous")
    refused(lambda: call(out_len=good["kv_len"]), "out_len", "kv_len")
    refused(lambda: call(out_len=torch.zeros(3, **I32)), "out_len")
    refused(lambda: call(out_table=torch.zeros(1, 2, **I32)), "out_table")
    refused(lambda: call(page_table=torch.zeros(2, 5)), "page_table")
    refused(lambda: call(weights=torch.zeros(2, 80)), "weights")
    refused(lambda: call(out_weights=torch.zeros(2, 2, 20, dtype=torch.float64)), "out_weights")
    refused(lambda: call(out_weights=torch.zeros(2, 1, 20).expand(2, 2, 20)), "out_weights", "overlap")
    whole = torch.zeros(2, 2, 81)
    refused(lambda: call(weights=whole[..., :80], out_weights=whole[..., 1:21]), "out_weights", "overlaps")
    refused(lambda: call(d_status=torch.zeros(1)), "d_status")


def test_blocks(guarded):
    c = cache()
    size = lw.lw_kv_summary_bytes(c)
    assert size == 3 * 2 * (2 * 64 + 16)
    good = dict(summary=torch.zeros(size, dtype=torch.uint8), q=rows(3, 4), q_start=torch.tensor([0, 1, 3], **I32),
                kv_len=torch.zeros(2, **I32), page_table=torch.zeros(2, 5, **I32), out=rows(3, 4),
                ws=torch.zeros(1000, dtype=torch.uint8), d_status=st())

    def call(**kw):
        a = {**good, **kw}
        lw.lw_kv_attention_blocks(c, a.pop("summary"), a.pop("q"), a.pop("q_start"), a.pop("kv_len"),
                                  a.pop("page_table"), a.pop("out"), a.pop("ws"), a.pop("d_status"),
                                  blocks=a.pop("blocks", 4), **a)

    refused(lambda: call(), "pages on cpu")
    refused(lambda: call(summary=torch.zeros(size - 1, dtype=torch.uint8)), "summary")
    refused(lambda: call(q=rows(3, 3)), "q", "multiple of 2")
    refused(lambda: call(out=rows(3, 4, dtype=torch.bfloat16)), "out", "bfloat16")
    refused(lambda: call(out=torch.zeros(1, 4, 64).expand(3, 4, 64)), "out", "overlap")
    refused(lambda: call(q_start=torch.zeros(2, **I32)), "q_start")
    refused(lambda: call(page_table=torch.zeros(5, 2, **I32).t()), "page_table", "contiguous")
    refused(lambda: call(lse=torch.zeros(11)), "lse")
    refused(lambda: call(chosen=torch.zeros(3, 2, 3, **I32)), "chosen")
    refused(lambda: call(chosen=torch.zeros(3, 2, 4, **I64)), "chosen")
    refused(lambda: call(blocks=1.0), "blocks")
    refused(lambda: call(recent=None), "recent")
    refused(lambda: call(d_status=None), "d_status")

    def sums(**kw):
        a = dict(summary=good["summary"], start=torch.zeros(2, **I32), kv_len=good["kv_len"],
                 page_table=good["page_table"], d_status=st())
        a.update(kw)
        lw.lw_kv_summarise(c, a["summary"], a["start"], a["kv_len"], a["page_table"], a["d_status"])

    refused(lambda: sums(), "pages on cpu")
    refused(lambda: sums(summary=good["summary"][:-1]), "summary")
    refused(lambda: sums(start=torch.zeros(3, **I32)), "start")
    refused(lambda: sums(start=torch.zeros(2, **I64)), "start", "int64")
    refused(lambda: sums(page_table=torch.zeros(3, 5, **I32)), "page_table")
    refused(lambda: sums(d_status=None), "d_status")


# ---- the C calls ------------------------------------------------------------

def view(**kw):
    v = lw.LwKvCache(FAKE, 10, 2, 64, 16, 0)
    for k, x in kw.items():
        setattr(v, k, x)
    return v


def status(fn, *args):
    lib = lw.load()
    r = getattr(lib, fn)(*args)
    return r, lib.lw_last_error().decode()


BAD_CACHES = [(dict(pages=None), INV), (dict(pages=FAKE + 8), INV), (dict(n_pages=0), SHP),
              (dict(n_pages=1 << 40), SHP), (dict(kv_heads=0), SHP), (dict(page_tokens=8), SHP),
              (dict(head_dim=80), UNS)]


def expect(call, cases):
    for kw, want in cases:
        r, msg = call(**kw)
        assert r == want and msg, (kw, r, msg)


def test_c_table():
    fields = ["rot", "scaling", "base", "factor", "old_length", "low", "high", "gain"]
    good = dict(rot=64, scaling=0, base=1e4, factor=1.0, old_length=0.0, low=0.0, high=0.0, gain=0.0)

    def call(first=0, n=4, table=FAKE, **kw):
        a = {**good, **kw}
        return status("lw_rotary_table", lw._ROTARY.pack(*(a[f] for f in fields)), first, n, table, None)

    nan, inf = float("nan"), float("inf")
    expect(call, [(dict(rot=0), SHP), (dict(rot=7), SHP), (dict(rot=130), SHP), (dict(scaling=5), UNS),
                  (dict(scaling=-1), UNS), (dict(base=1.0), INV), (dict(base=nan), INV), (dict(base=inf), INV),
                  (dict(scaling=1, factor=0.0), INV), (dict(scaling=2, factor=-1.0), INV),
                  (dict(scaling=3, factor=2.0), INV), (dict(scaling=4, factor=2.0, old_length=-1.0), INV),
                  (dict(scaling=3, factor=2.0, old_length=10.0, low=5.0), INV), (dict(gain=nan), INV),
                  (dict(first=-1), SHP), (dict(n=-1), SHP), (dict(first=1 << 31), SHP), (dict(n=1 << 40), SHP),
                  (dict(table=None), INV), (dict(table=FAKE + 2), INV)])
    assert status("lw_rotary_table", None, 0, 4, FAKE, None)[0] == INV
    assert call(n=0)[0] == lw.LW_OK


def test_c_rotary():
    row, q = (FAKE, 128, 64, 0, 0), (FAKE, 256, 64, 0, 0)
    good = dict(k=row, v=row, q=q, q_out=q, slots=FAKE, positions=FAKE, table=FAKE, rows=10, n=4, heads=4, rot=64,
                near=0)

    def call(**kw):
        a = {**good, **kw}
        return status("lw_kv_write_rotary", ctypes.byref(view()),
                      lw._KV_ROTATED.pack(*a["k"], *a["v"], *a["q"], *a["q_out"], a["slots"], a["positions"], a["table"],
                                          a["rows"], a["n"], a["heads"], a["rot"], a["near"], 0), None, None)

    for kw, want in BAD_CACHES:
        r, msg = status("lw_kv_write_rotary", ctypes.byref(view(**kw)), lw._KV_ROTATED.pack(*row * 4, *[0] * 9), None, None)
        assert r == want and msg
    def at(p, dtype=0):
        return (p, 128, 64, dtype, 0)
    expect(call, [
        (dict(k=at(0)), INV), (dict(v=at(0)), INV), (dict(k=at(FAKE + 2)), INV), (dict(k=at(FAKE, 7)), UNS),
        (dict(k=at(FAKE, 1)), INV), (dict(q=at(FAKE, 9)), UNS), (dict(q=at(FAKE, 1)), INV), (dict(q_out=at(0)), INV),
        (dict(q_out=at(FAKE, 2)), INV), (dict(q_out=at(FAKE + 1)), INV), (dict(slots=0), INV), (dict(positions=0), INV),
        (dict(positions=FAKE + 4), INV), (dict(table=0), INV), (dict(table=FAKE + 2), INV), (dict(rows=-1), SHP),
        (dict(rows=1 << 40), SHP), (dict(n=-1), INV), (dict(n=1 << 40), SHP), (dict(heads=0), SHP), (dict(rot=0), SHP),
        (dict(rot=63), SHP), (dict(rot=66), SHP), (dict(near=2), INV)])
    assert status("lw_kv_write_rotary", ctypes.byref(view()), None, None, None)[0] == INV
    assert call(n=0)[0] == lw.LW_OK


def test_c_weigh():
    fields = ["q", "qt", "qh", "lse", "q_start", "kv_len", "page_table", "table_stride", "q_tokens", "add", "ab", "ah",
              "weights", "wb", "wh", "keys", "table_width", "dtype", "batch", "q_heads", "max_q", "causal", "window",
              "scale"]
    good = dict(q=FAKE, qt=256, qh=64, lse=FAKE, q_start=FAKE, kv_len=FAKE, page_table=FAKE, table_stride=5,
                q_tokens=300, add=0, ab=0, ah=0, weights=FAKE, wb=160, wh=80, keys=80, table_width=5, dtype=0, batch=2,
                q_heads=4, max_q=2, causal=1, window=0, scale=0.125)
    need = lw.load().lw_kv_weigh_workspace_bytes(ctypes.byref(view()), 4, 300)
    assert need > 0 and lw.load().lw_kv_weigh_workspace_bytes(ctypes.byref(view()), 4, 2) == 0
    for heads, tokens in ((3, 10), (0, 10), (4, -1), (4, 1 << 40)):
        assert lw.load().lw_kv_weigh_workspace_bytes(ctypes.byref(view()), heads, tokens) == 0

    def call(v=None, ws=FAKE, ws_bytes=need, **kw):
        a = {**good, **kw}
        return status("lw_kv_weigh", ctypes.byref(view() if v is None else v),
                      lw._KV_WEIGHTS.pack(*(a[f] for f in fields)), ws, ws_bytes, None, None)

    for kw, want in BAD_CACHES:
        r, msg = call(view(**kw))
        assert r == want and msg, kw
    expect(call, [
        (dict(q=0), INV), (dict(lse=0), INV), (dict(q_start=0), INV), (dict(kv_len=0), INV), (dict(page_table=0), INV),
        (dict(weights=0), INV), (dict(q=FAKE + 2), INV), (dict(lse=FAKE + 1), INV), (dict(add=FAKE + 2), INV),
        (dict(weights=FAKE + 2), INV), (dict(dtype=3), UNS), (dict(batch=0), SHP), (dict(batch=70000), SHP),
        (dict(q_heads=3), SHP), (dict(q_tokens=-1), SHP), (dict(q_tokens=1 << 33), SHP), (dict(max_q=-1), INV),
        (dict(causal=2), INV), (dict(window=-1), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
        (dict(table_width=-1), SHP), (dict(table_width=1 << 30), SHP), (dict(table_stride=-1), SHP), (dict(keys=-1), INV),
        (dict(ws=0), INV), (dict(ws=FAKE + 8), INV), (dict(ws_bytes=need - 1), INV)])
    assert status("lw_kv_weigh", ctypes.byref(view()), None, FAKE, need, None, None)[0] == INV
    assert call(table_width=0)[0] == lw.LW_OK and call(keys=0)[0] == lw.LW_OK     # no key has a place


def test_c_evict():
    fields = ["weights", "wb", "wh", "keys", "kv_len", "page_table", "table_stride", "out_table", "out_stride", "out_len",
              "ow", "ob", "oh", "on", "kept", "table_width", "out_width", "batch", "keep", "first", "recent"]
    good = dict(weights=FAKE, wb=160, wh=80, keys=80, kv_len=FAKE, page_table=FAKE, table_stride=5, out_table=FAKE,
                out_stride=2, out_len=FAKE + 64, ow=FAKE, ob=40, oh=20, on=20, kept=FAKE, table_width=5, out_width=2,
                batch=2, keep=20, first=1, recent=4)

    def call(v=None, **kw):
        a = {**good, **kw}
        return status("lw_kv_evict", ctypes.byref(view() if v is None else v),
                      lw._KV_EVICTION.pack(*(a[f] for f in fields)), None, None)

    for kw, want in BAD_CACHES:
        r, msg = call(view(**kw))
        assert r == want and msg, kw
    expect(call, [
        (dict(weights=0), INV), (dict(kv_len=0), INV), (dict(page_table=0), INV), (dict(out_table=0), INV),
        (dict(out_len=0), INV), (dict(kept=0), INV), (dict(kept=FAKE + 2), INV), (dict(ow=FAKE + 1), INV),
        (dict(out_len=FAKE), INV), (dict(keep=0), INV), (dict(first=-1), INV), (dict(recent=-1), INV),
        (dict(first=10, recent=11), INV), (dict(keep=33), SHP), (dict(on=19), SHP), (dict(keys=-1), SHP),
        (dict(batch=0), SHP), (dict(batch=70000), SHP), (dict(table_width=-1), SHP), (dict(table_width=1 << 30), SHP),
        (dict(out_width=-1), SHP), (dict(out_width=1 << 30), SHP), (dict(table_stride=-1), SHP),
        (dict(out_stride=-1), SHP)])
    assert status("lw_kv_evict", ctypes.byref(view()), None, None, None)[0] == INV


def test_c_blocks():
    fields = ["q", "qt", "qh", "out", "ot", "oh", "lse", "q_start", "kv_len", "page_table", "table_stride", "q_tokens",
              "table_width", "dtype", "batch", "q_heads", "max_q", "causal", "window", "scale"]
    good = dict(q=FAKE, qt=256, qh=64, out=FAKE, ot=256, oh=64, lse=0, q_start=FAKE, kv_len=FAKE, page_table=FAKE,
                table_stride=5, q_tokens=3, table_width=5, dtype=0, batch=2, q_heads=4, max_q=0, causal=1, window=0,
                scale=0.125, summary=FAKE, chosen=0, blocks=4, first=1, recent=2)
    lib = lw.load()
    need = lib.lw_kv_blocks_workspace_bytes(ctypes.byref(view()), 4, 3, 5, 4)
    assert need > 0
    for bad in ((3, 3, 5, 4), (4, -1, 5, 4), (4, 40000, 5, 4), (4, 3, -1, 4), (4, 3, 50000, 4), (4, 3, 5, 0)):
        assert lib.lw_kv_blocks_workspace_bytes(ctypes.byref(view()), *bad) == 0

    def call(v=None, ws=FAKE, ws_bytes=need, **kw):
        a = {**good, **kw}
        return status("lw_kv_attention_blocks", ctypes.byref(view() if v is None else v),
                      lw._KV_ATTN.pack(*(a[f] for f in fields)),
                      lw._KV_BLOCKS.pack(a["summary"], a["chosen"], a["blocks"], a["first"], a["recent"], 0), ws, ws_bytes,
                      None, None)

    for kw, want in BAD_CACHES:
        r, msg = call(view(**kw))
        assert r == want and msg, kw
    expect(call, [
        (dict(q=0), INV), (dict(summary=0), INV), (dict(summary=FAKE + 8), INV), (dict(chosen=FAKE + 2), INV),
        (dict(causal=0), UNS), (dict(window=5), UNS), (dict(scale=0.0), UNS), (dict(scale=-1.0), UNS),
        (dict(scale=float("nan")), INV), (dict(blocks=0), INV), (dict(blocks=50000), INV), (dict(first=-1), INV),
        (dict(recent=0), INV), (dict(first=3), INV), (dict(table_width=50000), SHP), (dict(q_tokens=40000), SHP),
        (dict(q_heads=2 * 257), SHP), (dict(ws=0), INV), (dict(ws=FAKE + 8), INV), (dict(ws_bytes=need - 1), INV)])
    r, msg = call(view(n_pages=1 << 27))       # a head's share of a page as a page: too many of them
    assert r == SHP and msg
    assert call(q_tokens=0)[0] == lw.LW_OK
    assert status("lw_kv_attention_blocks", ctypes.byref(view()), None, None, FAKE, need, None, None)[0] == INV

    def sums(v=None, **kw):
        a = dict(summary=FAKE, start=FAKE, kv_len=FAKE, page_table=FAKE, stride=5, width=5, batch=2)
        a.update(kw)
        return status("lw_kv_summarise", ctypes.byref(view() if v is None else v), lw._KV_SUMMARIES.pack(*a.values()),
                      None, None)

    for kw, want in BAD_CACHES:
        r, msg = sums(view(**kw))
        assert r == want and msg, kw
    expect(sums, [(dict(summary=0), INV), (dict(summary=FAKE + 4), INV), (dict(start=0), INV), (dict(kv_len=0), INV),
                  (dict(page_table=0), INV), (dict(start=FAKE + 2), INV), (dict(batch=0), SHP), (dict(width=-1), SHP),
                  (dict(width=1 << 30), SHP), (dict(stride=-1), SHP)])
    assert status("lw_kv_summarise", ctypes.byref(view()), None, None, None)[0] == INV


def test_sizes_are_the_current_devices(monkeypatch):
    """A workspace is sized by the current device: with another one current than the cache's it is refused."""
    c = cache()
    c.index, c.device = 1, torch.device("cuda:1")
    now = [1]
    monkeypatch.setattr(lw, "_current_device", lambda: now[0])
    calls = (lambda: lw.lw_kv_weigh_workspace_bytes(c, 4, 300), lambda: lw.lw_kv_blocks_workspace_bytes(c, 4, 3, 5, 4))
    assert all(call() > 0 for call in calls)
    now[0] = 0
    for call in calls:
        refused(call, "current device")


def test_weights_that_lie_between_one_another(guarded):
    """Rows of one buffer that share no byte, as layers' weights beside one another: not refused (but for the device)."""
    c = cache()
    buf = torch.zeros(2, 3, 2, 80)                   # [batch][layer][kv_heads][keys]
    heads = torch.zeros(2, 2, 2, 80)                 # [batch][kv_heads][which][keys]
    wide = torch.zeros(2, 2, 120)
    i32 = dict(page_table=torch.zeros(2, 5, **I32), out_table=torch.zeros(2, 2, **I32))

    def weigh(weights, add_to):
        lw.lw_kv_weigh(c, rows(3, 4), torch.zeros(3, 4), torch.tensor([0, 1, 3], **I32), torch.zeros(2, **I32),
                       i32["page_table"], weights, torch.zeros(16, dtype=torch.uint8), st(), max_q=2, add_to=add_to)

    def evict(weights, out):
        lw.lw_kv_evict(c, weights, torch.zeros(2, **I32), i32["page_table"], i32["out_table"], torch.zeros(2, **I32), out,
                       torch.zeros(2, 2, 20, **I32), st(), keep=20)

    for call in (weigh, evict):
        for a, b in ((buf[:, 0], buf[:, 1]), (buf[:, 2], buf[:, 0]), (heads[:, :, 0], heads[:, :, 1])):
            refused(lambda: call(a, b), "pages on cpu")
        refused(lambda: call(buf[:, 0], buf[:, :2].flatten(1, 2)[:, 1:3]), "overlaps")     # a head of both
    refused(lambda: evict(wide[..., :80], wide[..., 80:]), "pages on cpu")                 # behind the weights, row by row
    refused(lambda: evict(wide[..., :80], wide[..., 79:]), "overlaps")


def test_positions_out_of_range(guarded, monkeypatch):
    """A first position that no 64-bit number holds is refused, not wrapped round to another one."""
    from test_kv_limits import on1
    monkeypatch.setattr(lw, "_current_device", lambda: 1)
    for first in (1 << 64, (1 << 64) + 5, -(1 << 70), 1 << 63, 1.5, "3", None):
        refused(lambda: lw.lw_rotary_table(on1(torch.zeros(4, 8)), first=first), "first")
    refused(lambda: lw.lw_rotary_table(on1(torch.zeros(4, 8)), base=10 ** 400), "base")
    refused(lambda: lw.lw_rotary_table(on1(torch.zeros(4, 8)), gain="x"), "gain")
