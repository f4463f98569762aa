"""Accumulated attention weight on the GPU, against the formula in 64 bits on the cached keys and the same lse.

Tolerance, normwise over a head's keys: a weight's exponent scale q.k - lse is a sum of terms of at most 60 in magnitude in all (scales times
code sums and middles times query sums, in these inputs), added in fp32 over some 16 steps, at worst
truncated: 60 * 16 * 2^-24 = 5.8e-5; fp32 queries' 22 bits add 60 * 2^-23 = 7e-6, the exponential 2^-21, the sum over
rows (all positive) as many 2^-24 as there are additions in a chain: 2000 / 8 here, 1.5e-5.  8e-5."""
import math

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from kv_plain import DEV, TYPES, filled, generator, i32, read, relative, scores, slots_of, spans, status
TOL = 8e-5


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def queries(gen, n, heads, dim, typ):
    return torch.randn(n, heads, dim, device=DEV, generator=gen).to(TYPES[typ])


def expected(cache, table, q, start, lens, lse, add, causal, window, scale):
    """fp64 [batch, kv_heads, max(lens)]; entries from a sequence's length on are NaN."""
    heads, group = cache.kv_heads, q.shape[1] // cache.kv_heads
    out = torch.full((len(lens), heads, max(max(lens), 1)), math.nan, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if not n:
            continue
        k, _ = read(cache, slots_of(table[b], range(n), cache.page_tokens))
        t0, t1 = start[b], start[b + 1]
        out[b, :, :n] = 0 if add is None else add[b, :, :n].double()
        if t1 > t0:
            see = spans(t1 - t0, n, causal, window)
            w = (scores(q[t0:t1], k, see, scale) - lse[t0:t1, :, None].double()).exp()
            w = torch.where(see[:, None], w, 0.0).view(t1 - t0, heads, group, n).sum((0, 2))
            out[b, :, :n] += w
    return out


def logsums(cache, table, q, start, lens, causal, window, scale):
    out = torch.full(q.shape[:2], -math.inf, device=DEV)
    for b, n in enumerate(lens):
        if n and start[b + 1] > start[b]:
            k, _ = read(cache, slots_of(table[b], range(n), cache.page_tokens))
            see = spans(start[b + 1] - start[b], n, causal, window)
            out[start[b]:start[b + 1]] = scores(q[start[b]:start[b + 1]], k, see, scale).logsumexp(-1).float()
    return out


def weigh(cache, table, q, lse, start, lens, weights, st, **kw):
    need = lw.lw_kv_weigh_workspace_bytes(cache, q.shape[1], q.shape[0])
    ws = torch.randint(0, 256, (max(need, 16),), dtype=torch.uint8, device=DEV)    # (holds nothing before a call)
    lw.lw_kv_weigh(cache, q, lse, i32(start), i32(lens), table, weights, ws, st, **kw)
    torch.cuda.synchronize()


CASES = [   # query tokens, lens, q heads, kv heads, dim, page, causal, window
    ([1], [37], 32, 8, 128, 64, True, 0), ([1, 1, 1], [1, 16, 17], 4, 2, 64, 16, True, 0),
    ([1, 0, 5, 2], [4097, 100, 700, 0], 6, 2, 96, 48, True, 0), ([7, 3], [333, 20], 8, 1, 128, 16, False, 0),
    ([1, 4], [2000, 300], 3, 3, 64, 256, True, 129), ([40, 90], [41, 1200], 8, 2, 128, 64, True, 0),
    ([300], [300], 4, 1, 64, 32, True, 50), ([17, 130], [600, 130], 12, 4, 96, 16, False, 100),
    ([500, 3], [900, 2], 8, 8, 128, 128, True, 0), ([5], [3], 4, 2, 64, 16, True, 0),
    ([700], [2100], 8, 2, 96, 48, True, 0), ([257, 260, 1], [257, 1000, 500], 16, 2, 64, 64, True, 200),
]


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_weigh(typ, case):
    ts, lens, hq, h, dim, page, causal, window = case
    gen, st = generator(sum(lens) + hq), status()
    cache, table, _ = filled(gen, lens, h, dim, page)
    start = [sum(ts[:i]) for i in range(len(ts) + 1)]
    q, scale = queries(gen, start[-1], hq, dim, typ), 1.2 / math.sqrt(dim)
    lse = logsums(cache, table, q, start, lens, causal, window, scale)
    keys = max(max(lens), 1)
    store = torch.full((len(lens), h, keys + 3), 11.0, device=DEV)
    w, add = store[..., :keys], torch.rand(len(lens), h, keys, device=DEV, generator=gen)
    kw = dict(scale=scale, causal=causal, window=window, max_q=max(ts))
    for given in (None, add, "itself"):
        if given == "itself":
            given = w
        want = expected(cache, table, q, start, lens, lse, given, causal, window, scale)
        weigh(cache, table, q, lse, start, lens, w, st, add_to=given, **kw)
        for b, n in enumerate(lens):
            for i in range(h):
                assert relative(w[b, i, :n], want[b, i, :n]) <= TOL, (b, i)
            assert bool((store[b, :, n:] == 11).all())
    assert int(st) == 0
    # the hint changes nothing but the kernel; the same call twice gives the same bits
    first = None
    for hint in (0, 1, 10 ** 6):
        for _ in range(2):
            weigh(cache, table, q, lse, start, lens, w, st, **{**kw, "max_q": hint})
            got = torch.where(torch.isnan(want), 0.0, w)
            assert first is None or relative(got, first) <= TOL
            assert _ == 0 or torch.equal(got, last)
            last, first = got.clone(), got.clone() if first is None else first


def test_attention_hands_its_lse_on():
    """The weights of lw_kv_attention's rows add up to one a row."""
    gen, st = generator(8), status()
    for typ in ("fp32", "bf16"):
        lens, ts, hq, h, dim = [3000, 700], [1, 6], 8, 2, 128
        cache, table, _ = filled(gen, lens, h, dim, 64)
        q = queries(gen, 7, hq, dim, typ)
        lse, out = torch.empty(7, hq, device=DEV), torch.empty_like(q)
        ws = torch.zeros(lw.lw_kv_workspace_bytes(cache, hq, 7, 2), dtype=torch.uint8, device=DEV)
        lw.lw_kv_attention(cache, q, i32([0, 1, 7]), i32(lens), table, out, ws, st, max_q=6, lse=lse)
        w = torch.empty(2, h, 3000, device=DEV)
        weigh(cache, table, q, lse, [0, 1, 7], lens, w, st, max_q=6)
        assert int(st) == 0
        tol = 1e-4 if typ == "fp32" else 1e-2       # (lse's own error, by the type's operands)
        for b, n in enumerate(lens):
            for i in range(h):
                assert abs(float(w[b, i, :n].double().sum()) / (ts[b] * hq / h) - 1) < tol


@pytest.mark.parametrize("tokens", [1, 200])
@pytest.mark.parametrize("typ", ["fp32", "bf16"])
def test_queries_of_any_magnitude_and_odd_strides(typ, tokens):
    gen, st = generator(9), status()
    cache, table, _ = filled(gen, [500], 2, 128, 16)
    q0 = torch.randn(tokens, 4, 128, device=DEV, generator=gen)
    for mag in (1e-12, 1e-3, 1e4, 1e20):
        q = torch.zeros(tokens, 5, 131, dtype=TYPES[typ], device=DEV)[:, 1:, 2:130]
        q.copy_(q0 * mag)
        scale = 0.09 / mag
        lse = logsums(cache, table, q, [0, tokens], [500], True, 0, scale)
        w = torch.empty(1, 2, 500, device=DEV)
        weigh(cache, table, q, lse, [0, tokens], [500], w, st, scale=scale, max_q=tokens)
        assert relative(w, expected(cache, table, q, [0, tokens], [500], lse, None, True, 0, scale)) <= TOL
    assert int(st) == 0


@pytest.mark.parametrize("tokens", [2, 300])
def test_negative_scale_and_rows_that_see_nothing(tokens):
    """lse = -inf where a row sees no key: it weighs nothing, whatever else it holds."""
    gen, st = generator(10), status()
    cache, table, _ = filled(gen, [tokens // 2], 1, 64, 16)
    q = queries(gen, tokens, 2, 64, "fp16")
    n, start = tokens // 2, [0, tokens]
    lse = logsums(cache, table, q, start, [n], True, 0, -0.2)
    assert bool(torch.isinf(lse[0]).all())
    w = torch.empty(1, 1, n, device=DEV)
    weigh(cache, table, q, lse, start, [n], w, st, scale=-0.2, max_q=tokens)
    assert relative(w, expected(cache, table, q, start, [n], lse, None, True, 0, -0.2)) <= TOL


@pytest.mark.parametrize("tokens", [3, 150])
def test_nan(tokens):
    """A NaN key is a NaN weight; a row whose lse is one, in the keys that it sees."""
    gen, st = generator(11), status()
    n, page = 400, 32
    cache, table, _ = filled(gen, [n], 2, 64, page)
    k, v = torch.zeros(1, 2, 64, device=DEV), torch.zeros(1, 2, 64, device=DEV)
    q = queries(gen, tokens, 2, 64, "bf16")
    lse = logsums(cache, table, q, [0, tokens], [n], True, 0, 0.1)
    k[0, 1, 7] = math.nan
    lw.lw_kv_write(cache, k, v, slots_of(table[0], [100], page), st)
    w = torch.empty(1, 2, n, device=DEV)
    weigh(cache, table, q, lse, [0, tokens], [n], w, st, scale=0.1, max_q=tokens)
    want = expected(cache, table, q, [0, tokens], [n], lse, None, True, 0, 0.1)
    assert torch.equal(torch.isnan(w), torch.isnan(want)) and int(torch.isnan(w).sum()) == 1
    lse[tokens // 2, 0] = math.nan
    weigh(cache, table, q, lse, [0, tokens], [n], w, st, scale=0.1, max_q=tokens)
    want = expected(cache, table, q, [0, tokens], [n], lse, None, True, 0, 0.1)
    assert torch.equal(torch.isnan(w), torch.isnan(want))


@pytest.mark.parametrize("tokens", [2, 200])
def test_pages_and_sequences_that_are_not_there(tokens):
    gen, st = generator(12), status()
    lens, page = [400, 300], 16
    cache, table, _ = filled(gen, lens, 2, 128, page)
    q = queries(gen, 2 * tokens, 4, 128, "bf16")
    start = [0, tokens, 2 * tokens]
    lse = logsums(cache, table, q, start, lens, True, 0, 0.1)
    want = expected(cache, table, q, start, lens, lse, None, True, 0, 0.1)
    bad = table.clone()
    bad[0, 3], bad[1, 0] = -7, cache.n_pages
    w = torch.full((2, 2, 400), 3.0, device=DEV)
    weigh(cache, bad, q, lse, start, lens, w, st, scale=0.1, max_q=tokens)
    assert int(st) == lw.LW_DEV_BAD_PAGE
    want[0, :, 48:64] = 0
    want[1, :, :16] = 0
    for b, n in enumerate(lens):
        assert relative(w[b, :, :n], want[b, :, :n]) <= TOL
    st = status()        # rows shorter than a sequence
    w.fill_(3.0)
    weigh(cache, table, q, lse, start, lens, w[..., :350], st, scale=0.1, max_q=tokens)
    assert int(st) == lw.LW_DEV_BAD_SEQ and bool((w[..., 350:] == 3).all())
    want = expected(cache, table, q, start, lens, lse, None, True, 0, 0.1)
    assert relative(w[0, :, :350], want[0, :, :350]) <= TOL
    st = status()        # query ranges that are none: no weight from them, add_to kept
    w.fill_(3.0)
    weigh(cache, table, q, lse, [0, 5 * tokens, 2 * tokens], lens, w, st, scale=0.1, max_q=tokens, add_to=w)
    assert int(st) == lw.LW_DEV_BAD_SEQ and bool((w[0] == 3).all()) and bool((w[1] == 3).all())


def test_two_streams_and_replay():
    """Calls of two streams at once, each captured with a workspace of its own."""
    gen = generator(13)
    jobs = []
    for i, tokens in enumerate((1, 400)):
        st, side = status(), torch.cuda.Stream()
        lens = [1500 + 100 * i]
        cache, table, _ = filled(gen, lens, 2, 128, 64)
        q = queries(gen, tokens, 8, 128, "bf16")
        lse = logsums(cache, table, q, [0, tokens], lens, True, 0, 0.1)
        want = expected(cache, table, q, [0, tokens], lens, lse, None, True, 0, 0.1)
        w = torch.zeros(1, 2, lens[0], device=DEV)
        ws = torch.empty(max(16, lw.lw_kv_weigh_workspace_bytes(cache, 8, tokens)), dtype=torch.uint8, device=DEV)
        at, n = i32([0, tokens]), i32(lens)
        torch.cuda.synchronize()
        g = lw.StepGraph(side)
        with g.capture():
            lw.lw_kv_weigh(cache, q, lse, at, n, table, w, ws, st, max_q=tokens, scale=0.1, add_to=w)
        jobs.append((g, w, want, st, (cache, table, q, lse, ws, at, n)))
    for _ in range(3):
        for g, *_ in jobs:
            g.launch()
    torch.cuda.synchronize()
    for _, w, want, st, _ in jobs:
        assert int(st) == 0 and relative(w, 3 * want) <= TOL


def test_many_sequences_of_many_rows():
    """More heads of sequences than CTAs: one takes several units of 128 keys, under a table far wider than most
    sequences are long; and the same rows by way of the few-row kernel."""
    gen, st = generator(14), status()
    ts = [66 + i % 5 for i in range(80)]
    lens = [t + (37 * i) % 500 for i, t in enumerate(ts)]
    cache, table, free = filled(gen, lens, 16, 64, 32)
    table = torch.cat([table, torch.full((80, 40), -1, dtype=torch.int32, device=DEV)], 1)
    start = [sum(ts[:i]) for i in range(81)]
    q = queries(gen, start[-1], 16, 64, "bf16")
    lse = logsums(cache, table, q, start, lens, True, 0, 0.125)
    want = expected(cache, table, q, start, lens, lse, None, True, 0, 0.125)
    keys = table.shape[1] * 32
    for hint in (70, 1):
        w = torch.full((80, 16, keys), 9.0, device=DEV)
        weigh(cache, table, q, lse, start, lens, w, st, scale=0.125, max_q=hint)
        for b, n in enumerate(lens):
            assert relative(w[b, :, :n], want[b, :, :n]) <= TOL, (hint, b)
            assert bool((w[b, :, n:] == 9).all())
    assert int(st) == 0


def test_no_queries():
    """Sequences without query tokens: what was there, or zeros."""
    gen, st = generator(15), status()
    cache, table, _ = filled(gen, [70, 0], 2, 64, 16)
    q, lse = queries(gen, 0, 4, 64, "fp32"), torch.empty(0, 4, device=DEV)
    w = torch.rand(2, 2, 75, device=DEV, generator=gen)
    had = w.clone()
    weigh(cache, table, q, lse, [0, 0, 0], [70, 0], w, st, max_q=0, add_to=w)
    assert torch.equal(w, had)
    weigh(cache, table, q, lse, [0, 0, 0], [70, 0], w, st, max_q=0)
    assert not bool(w[0, :, :70].any()) and torch.equal(w[0, :, 70:], had[0, :, 70:]) and torch.equal(w[1], had[1])
    assert int(st) == 0


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
@pytest.mark.parametrize("ts", [[1, 0, 3], [60, 0, 700], [400, 0, 5]], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_pages_that_no_row_sees_are_not_needed(ts, causal, typ):
    """Pages behind the window, and those of a sequence without query tokens, are freed: attention with the same
    arguments does not read them, and neither do its weights.  What was there stays, or is 0."""
    gen, st, lens, page, window = generator(16 + sum(ts)), status(), [3000, 900, 2500], 16, 129
    cache, table, _ = filled(gen, lens, 2, 64, page)
    start = [sum(ts[:i]) for i in range(4)]
    q = queries(gen, start[-1], 8, 64, typ)
    freed = table.clone()
    first = [max(0, n - t - window + 1) if t else n for n, t in zip(lens, ts)]      # the first key that a row sees
    for b in range(3):
        freed[b, :first[b] // page if ts[b] else None] = -1
    kw = dict(max_q=max(ts), causal=causal, window=window, scale=0.125)
    lse, out = torch.empty(start[-1], 8, device=DEV), torch.empty_like(q)
    ws = torch.zeros(lw.lw_kv_workspace_bytes(cache, 8, start[-1], 3), dtype=torch.uint8, device=DEV)
    lw.lw_kv_attention(cache, q, i32(start), i32(lens), freed, out, ws, st, lse=lse, **kw)
    assert int(st) == 0
    lse = logsums(cache, table, q, start, lens, causal, window, 0.125)
    add = torch.rand(3, 2, 3000, device=DEV, generator=gen)
    for given in (None, add):
        want = expected(cache, table, q, start, lens, lse, given, causal, window, 0.125)
        for hint in (max(ts), 1):
            w = torch.full((3, 2, 3000), 7.0, device=DEV)
            weigh(cache, freed, q, lse, start, lens, w, st, add_to=given, **{**kw, "max_q": hint})
            assert int(st) == 0
            for b, n in enumerate(lens):
                assert relative(w[b, :, :n], want[b, :, :n]) <= TOL, (b, hint)
                unseen = torch.zeros_like(w[b, :, :first[b]]) if given is None else given[b, :, :first[b]]
                assert torch.equal(w[b, :, :first[b]], unseen) and bool((w[b, :, n:] == 7).all())
    # the page of the first key that is seen is needed
    gone = freed.clone()
    gone[0, first[0] // page] = -1
    weigh(cache, gone, q, lse, start, lens, w, st, **kw)
    assert int(st) == lw.LW_DEV_BAD_PAGE


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 30, 300])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_keys_of_any_magnitude(typ, tokens, dim):
    """Keys from the smallest that fp16 scales hold to the format's limit, with queries that bring the scores to unit
    spread; in the last sequence large and small keys by turns of 100, each part's weights looked at alone.
    A product's keys keep 2^-21 of the largest of a unit's, some 5 times the usual one: with terms of 12 in all at
    most, 12 (16 2^-24 + 5 2^-21 + 2^-23) = 4e-5 beside the exponential's and the sums' 1.6e-5."""
    gen, st, n, page = generator(17), status(), 700, 16
    mags = (1e-5, 1e-3, 0.03, 1.0, 12000.0, None)
    cache, table, _ = filled(gen, [n] * 6, 2, dim, page)
    k = torch.randn(6, n, 2, dim, device=DEV, generator=gen)
    q = torch.randn(6, tokens, 4, dim, device=DEV, generator=gen)
    for b, mag in enumerate(mags):
        if mag is None:
            k[b] *= torch.where(torch.arange(n, device=DEV) // 100 % 2 == 0, 1.0, 1e-3)[:, None, None]
        else:
            k[b], q[b] = k[b].clamp(-5, 5) * mag, q[b] / mag
        lw.lw_kv_write(cache, k[b], k[b], slots_of(table[b], range(n), page), st)
    q, start, lens = q.flatten(0, 1).to(TYPES[typ]), [tokens * b for b in range(7)], [n] * 6
    scale = 0.7 / math.sqrt(dim)
    lse = logsums(cache, table, q, start, lens, True, 0, scale)
    want = expected(cache, table, q, start, lens, lse, None, True, 0, scale)
    w = torch.empty(6, 2, n, device=DEV)
    for hint in (tokens, 1):
        weigh(cache, table, q, lse, start, lens, w, st, scale=scale, max_q=hint)
        for b in range(6):
            for at in range(0, n, 100):
                part = slice(at, at + 100)
                assert relative(w[b, :, part], want[b, :, part]) <= TOL, (b, at, hint)
    assert int(st) == 0


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 1000, 4000])
def test_units_of_one_cta(typ, dim, window):
    """A long sequence's units of 128 keys are more than the CTAs of its heads: each takes several, the first of them
    without a row under a window."""
    gen, st, n, heads, tokens = generator(18), status(), 9000, 8, 300
    cache, table, _ = filled(gen, [n], heads, dim, 64)
    q, scale = queries(gen, tokens, heads, dim, typ), 1 / math.sqrt(dim)
    lse = logsums(cache, table, q, [0, tokens], [n], True, window, scale)
    add = torch.rand(1, heads, n, device=DEV, generator=gen)
    want = expected(cache, table, q, [0, tokens], [n], lse, add, True, window, scale)
    w = torch.empty(1, heads, n, device=DEV)
    for _ in range(2):
        weigh(cache, table, q, lse, [0, tokens], [n], w, st, scale=scale, max_q=tokens, add_to=add, window=window)
        for h in range(heads):
            assert relative(w[0, h], want[0, h]) <= TOL
    assert int(st) == 0
