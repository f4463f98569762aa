"""Eviction on the GPU: the kept keys against a sort with the same rules, the moved tokens bit for bit, and every
other token of the pool as it was.  Nothing is computed but comparisons: all exact."""
import math

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from kv_plain import DEV, filled, generator, i32, read, read_all, slots_of, status


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def choose(w, n, keep, first, recent):
    """Kept keys of one head, ascending: by a sort in Python."""
    if n <= keep:
        return list(range(n))
    always = set(range(first)) | set(range(n - recent, n))
    others = [j for j in range(n) if j not in always]
    others.sort(key=lambda j: (-math.inf if w[j] != w[j] else -w[j], w[j] == w[j], j))
    # (a NaN before an infinity)
    return sorted(always | set(others[:keep - len(always)]))


def weights(gen, batch, heads, keys, kind):
    w = torch.rand(batch, heads, keys, device=DEV, generator=gen) ** 6
    if kind == "ties":
        w = torch.floor(w * 4) / 4
        w[..., ::7] = -0.0
    elif kind == "odd":
        w[..., 1::5] *= -3.0
        w[..., 3::11] = math.inf
        w[..., 4::13] = math.nan
        w[..., 6::17] = -math.inf
    elif kind == "equal":
        w.fill_(0.25)
    return w


CASES = [   # lens, heads, dim, page, keep, first, recent
    ([37], 1, 64, 16, 20, 1, 4), ([0, 1, 16, 17, 100], 2, 128, 16, 16, 0, 0), ([333, 200], 3, 96, 48, 97, 4, 33),
    ([1000], 2, 128, 64, 999, 0, 0), ([500, 64], 1, 64, 256, 1, 0, 0), ([500, 64], 1, 96, 32, 64, 30, 34),
    ([700, 3, 700], 2, 128, 32, 300, 0, 300), ([2600], 1, 128, 64, 2200, 4, 100), ([5003, 2], 8, 64, 16, 1234, 33, 0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind", ["plain", "ties", "odd", "equal"])
@pytest.mark.parametrize("place", ["apart", "in place"])
def test_evict(case, kind, place):
    lens, heads, dim, page, keep, first, recent = case
    batch, gen, st = len(lens), generator(sum(lens) + keep), status()
    to = -(-keep // page)
    cache, table, free = filled(gen, lens, heads, dim, page, batch * to)
    n = max(lens) + 5
    store = weights(gen, batch, heads, n + 3, kind)
    w = store[..., :n]                       # rows that are strided
    host = w.cpu().tolist()
    before = read_all(cache)
    out_table = table if place == "in place" else free[:batch * to].view(batch, to).contiguous()
    if place == "in place" and table.shape[1] * page < keep:
        pytest.skip("fewer pages than the call asks for")
    out_len, kept = i32([7] * batch), torch.full((batch, heads, keep), 9, dtype=torch.int32, device=DEV)
    ow = w if place == "in place" else torch.full((batch, heads, keep + 2), 5.0, device=DEV)
    first_w, behind = w.clone(), store[..., n:].clone().view(torch.int32)
    kv_len = i32(lens)
    lw.lw_kv_evict(cache, w, kv_len, table, out_table, out_len, ow, kept, st, keep=keep, first=first, recent=recent)
    torch.cuda.synchronize()
    assert int(st) == 0
    want = before.clone()
    for b, length in enumerate(lens):
        m = min(length, keep)
        assert int(out_len[b]) == m
        for h in range(heads):
            at = choose(host[b][h], length, keep, first, recent)
            assert kept[b, h].tolist() == at + [-1] * (keep - m)
            ref = first_w[b, h].clone() if place == "in place" else torch.full((keep + 2,), 5.0, device=DEV)
            ref[m:length] = 0
            ref[:m] = first_w[b, h, at]
            assert torch.equal(ow[b, h].clone().view(torch.int32), ref.view(torch.int32))
            if m:
                src, dst = slots_of(table[b], at, page), slots_of(out_table[b], range(m), page)
                want[:, dst, h] = before[:, src, h]
    assert torch.equal(read_all(cache), want)
    assert torch.equal(store[..., n:].clone().view(torch.int32), behind)


def test_no_weights_out_and_pages_that_are_not_there():
    gen, st = generator(1), status()
    cache, table, free = filled(gen, [200], 2, 64, 16, 4)
    w = weights(gen, 1, 2, 200, "plain")
    before = read_all(cache)
    kept, out_len = torch.empty(1, 2, 50, dtype=torch.int32, device=DEV), i32([0])
    out_table = free[:4].view(1, 4).clone()
    good = out_table.clone()
    out_table[0, 1], bad = cache.n_pages, table.clone()
    bad[0, 12] = -5
    lw.lw_kv_evict(cache, w, i32([200]), bad, out_table, out_len, None, kept, st, keep=50, first=0, recent=8)
    assert int(st) == lw.LW_DEV_BAD_PAGE
    after = read_all(cache)
    for h in range(2):
        at = choose(w[0, h].tolist(), 200, 50, 0, 8)
        assert kept[0, h].tolist() == at
        for i, j in enumerate(at):
            dst = int(slots_of(good[0], [i], 16))
            if 16 <= i < 32 or j >= 192:
                assert torch.equal(after[:, dst, h], before[:, dst, h])      # not moved
            else:
                src = int(slots_of(table[0], [j], 16))
                assert torch.equal(after[:, dst, h], before[:, src, h])
    st = status()
    lw.lw_kv_evict(cache, w[..., :100], i32([200]), table, good, out_len, None, kept, st, keep=50)
    assert int(st) == lw.LW_DEV_BAD_SEQ and int(kept.max()) < 100
    st = status()
    lw.lw_kv_evict(cache, w, i32([-3]), table, good, out_len, None, kept, st, keep=50)
    assert int(st) == lw.LW_DEV_BAD_SEQ and int(out_len) == 0 and int(kept.max()) == -1


def test_replayed():
    """One captured call on new weights and lengths; twice on the same (already short) sequence in place."""
    gen, st = generator(2), status()
    cache, table, _ = filled(gen, [900, 400], 4, 128, 64)
    w, kv_len = weights(gen, 2, 4, 900, "plain"), i32([900, 400])
    kept, out_len = torch.empty(2, 4, 300, dtype=torch.int32, device=DEV), i32([0, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = lw.StepGraph(side)
    with g.capture():
        lw.lw_kv_evict(cache, w, kv_len, table, table, out_len, w, kept, st, keep=300, first=2, recent=50)
    for _ in range(3):
        host, lens, before = w.clone(), kv_len.tolist(), read_all(cache)
        torch.cuda.synchronize()
        g.launch()
        torch.cuda.synchronize()
        after = read_all(cache)
        for b in range(2):
            for h in range(4):
                at = choose(host[b, h].tolist(), lens[b], 300, 2, 50)
                assert kept[b, h].tolist()[:len(at)] == at
                assert torch.equal(after[:, slots_of(table[b], range(len(at)), 64), h],
                                   before[:, slots_of(table[b], at, 64), h])
                assert torch.equal(w[b, h, :len(at)], host[b, h, at])
        kv_len.copy_(out_len)
    assert int(st) == 0


@pytest.mark.parametrize("kind", ["plain", "ties", "equal"])
def test_more_keys_than_shared_memory_holds(kind):
    """400000 keys of one head: eight CTAs' stretches of 50000 are read again instead of kept."""
    gen, st, n, keep = generator(3), status(), 400000, 1500
    cache, table, free = filled(gen, [n], 1, 64, 256, 6)
    w = weights(gen, 1, 1, n, kind)
    kept, out_len = torch.empty(1, 1, keep, dtype=torch.int32, device=DEV), i32([0])
    out, to = torch.empty(1, 1, keep, device=DEV), free[:6].view(1, 6).contiguous()
    before = read(cache, slots_of(table[0], range(n), 256))
    lw.lw_kv_evict(cache, w, i32([n]), table, to, out_len, out, kept, st, keep=keep, first=7, recent=100)
    at = choose(w[0, 0].tolist(), n, keep, 7, 100)
    assert int(st) == 0 and kept[0, 0].tolist() == at and int(out_len) == keep
    assert torch.equal(out[0, 0], w[0, 0, at])
    now = read(cache, slots_of(to[0], range(keep), 256))
    assert all(torch.equal(x, y[at]) for x, y in zip(now, before))
