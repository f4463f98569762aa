"""Block-sparse attention on the GPU: summaries and chosen pages against the definition (exact: its sums are whole
numbers, its fp32 steps are fixed), the attention over the chosen pages against a softmax in 64 bits, with the
tolerances of lw_kv_attention (1e-2 + 2^-8 in bf16, 7.6e-5 + 2^-11 in fp16, 7.6e-5 in fp32)."""
import math

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from kv_plain import DEV, TYPES, filled, generator, i32, keys_values, read, relative, slots_of, status
TOL = {"fp32": 7.6e-5, "fp16": 7.6e-5 + 2.0 ** -11, "bf16": 1e-2 + 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def coded(x, top):
    """rint(fl(x fl(127 fl(1 / top)))), 0 where top is too small."""
    one = torch.ones_like(top)
    inv = torch.where(top > 2.0 ** -100, 127.0 * (one / top), torch.zeros_like(top))
    return torch.round(x * inv), top * torch.full_like(top, 1 / 127)


def summary_of(cache, row, n):
    """hi, lo codes [blocks, heads, D] and steps [blocks, heads] of one sequence's pages."""
    page = cache.page_tokens
    k, _ = read(cache, slots_of(row, range(n), page))
    nb = -(-n // page)
    k = torch.cat([k, k[-1:].expand(nb * page - n, *k.shape[1:])]).view(nb, page, *k.shape[1:])
    hi, lo = k.amax(1), k.amin(1)
    top = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    (chi, step), (clo, _) = coded(hi, top[..., None]), coded(lo, top[..., None])
    return chi, clo, step[..., 0]


def fields(cache, summary, pages):
    d = cache.head_dim
    rec = summary.view(cache.n_pages, cache.kv_heads, 2 * d + 16)[pages.long()]
    return (rec[..., :d].view(torch.int8).float(), rec[..., d:2 * d].view(torch.int8).float(),
            rec[..., 2 * d:2 * d + 4].contiguous().view(torch.float32)[..., 0])


def chosen_by(scores, nb, blocks, first, recent):
    if nb <= blocks:
        return list(range(nb))
    always = set(range(first)) | set(range(nb - recent, nb))
    others = sorted((j for j in range(nb) if j not in always),
                    key=lambda j: (-math.inf if scores[j] != scores[j] else -scores[j], j))
    return sorted(always | set(others[:blocks - len(always)]))


def attend(cache, summary, q, start, lens, table, st, blocks, first, recent, out=None, ws=None, **kw):
    out = torch.full_like(q, 5.0) if out is None else out
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    chosen = torch.full((q.shape[0], cache.kv_heads, blocks), -9, dtype=torch.int32, device=DEV)
    if ws is None:
        ws = torch.zeros(lw.lw_kv_blocks_workspace_bytes(cache, q.shape[1], q.shape[0], table.shape[1], blocks),
                         dtype=torch.uint8, device=DEV)
    lw.lw_kv_attention_blocks(cache, summary, q, i32(start), i32(lens), table, out, ws, st, blocks=blocks, first=first,
                              recent=recent, lse=lse, chosen=chosen, **kw)
    torch.cuda.synchronize()
    return out, lse, chosen


def check(cache, q, start, lens, table, blocks, first, recent, scale, got, tol, skip=()):
    out, lse, chosen = got
    page, heads, group = cache.page_tokens, cache.kv_heads, q.shape[1] // cache.kv_heads
    for b, n in enumerate(lens):
        T = start[b + 1] - start[b]
        if not n:
            assert bool((out[start[b]:start[b + 1]] == 0).all()) and bool((lse[start[b]:start[b + 1]] == -math.inf).all())
            continue
        chi, clo, step = summary_of(cache, table[b], n)
        k, v = (x.double() for x in read(cache, slots_of(table[b], range(n), page)))
        for t in range(T):
            i, pos = start[b] + t, n - T + t
            nb = pos // page + 1
            for h in range(heads):
                rows = q[i, h * group:(h + 1) * group]
                if pos < 0:
                    assert chosen[i, h].tolist() == [-1] * blocks
                    assert bool((out[i, h * group:(h + 1) * group] == 0).all())
                    continue
                c, u = coded(rows.float(), rows.float().abs().amax(-1, keepdim=True))
                dot = torch.maximum(c[:, None] * chi[:nb, h], c[:, None] * clo[:nb, h]).double().sum(-1).float()
                score = (dot * u).amax(0) * step[:nb, h]
                at = chosen_by(score.tolist(), nb, blocks, first, recent)
                assert chosen[i, h].tolist() == at + [-1] * (blocks - len(at)), (b, t, h)
                key = torch.tensor([j for x in at for j in range(x * page, min(x * page + page, pos + 1))], device=DEV)
                s = rows.double() @ k[key, h].T * scale
                assert relative(out[i, h * group:(h + 1) * group], s.softmax(-1) @ v[key, h]) <= tol
                assert float((lse[i, h * group:(h + 1) * group] - s.logsumexp(-1)).abs().max()) <= 4 * tol + 1e-4


CASES = [   # query tokens, lens, q heads, kv heads, dim, page, blocks, first, recent
    ([1], [37], 32, 8, 128, 64, 4, 1, 1), ([1], [4097], 32, 8, 128, 64, 16, 1, 2),
    ([2, 0, 1, 3], [700, 90, 1, 333], 6, 2, 96, 48, 3, 0, 1), ([5, 1], [1000, 17], 4, 4, 64, 16, 9, 2, 3),
    ([1, 4], [0, 2], 2, 1, 64, 16, 2, 1, 1), ([3], [900], 16, 1, 128, 32, 5, 0, 5),
    ([1, 1], [3000, 2000], 40, 1, 64, 16, 33, 1, 2), ([8], [520], 3, 3, 96, 256, 1, 0, 1),
    ([1], [5000], 8, 2, 128, 16, 300, 4, 10),
]


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_blocks(typ, case):
    ts, lens, hq, h, dim, page, blocks, first, recent = case
    gen, st = generator(sum(lens) + hq), status()
    cache, table, _ = filled(gen, lens, h, dim, page)
    start = [sum(ts[:i]) for i in range(len(ts) + 1)]
    q = torch.randn(start[-1], hq, dim, device=DEV, generator=gen).to(TYPES[typ])
    summary = torch.randint(0, 256, (lw.lw_kv_summary_bytes(cache),), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([-4] * len(lens)), i32(lens), table, st)
    for b, n in enumerate(lens):
        if n:
            want = summary_of(cache, table[b], n)
            got = fields(cache, summary, table[b, :-(-n // page)])
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    for scale in (1 / math.sqrt(dim), 0.3):
        got = attend(cache, summary, q, start, lens, table, st, blocks, first, recent, scale=scale)
        check(cache, q, start, lens, table, blocks, first, recent, scale, got, TOL[typ])
    assert int(st) == 0
    # rows in a wider buffer, on no 16-byte boundary: the same bits
    for pad, at in ((0, 0), (3, 1)):
        wide = torch.zeros(start[-1], hq + 2, dim + pad, dtype=TYPES[typ], device=DEV)
        qs = wide[:, 1:hq + 1, at:at + dim]
        qs.copy_(q)
        os = torch.full_like(wide, 4.0)
        again = attend(cache, summary, qs, start, lens, table, st, blocks, first, recent, scale=0.3,
                       out=os[:, 1:hq + 1, at:at + dim])
        assert all(torch.equal(x, y) for x, y in zip(again, got))
        assert bool((os[:, 0] == 4).all()) and bool((os[:, hq + 1] == 4).all())


def test_summaries_step_by_step():
    """Tokens written one by one, and only the pages that they touch summed up again."""
    gen, st = generator(2), status()
    lens = [30, 64]
    cache, table, free = filled(gen, lens, 2, 64, 32, 4)
    table = torch.cat([table, free[:4].view(2, 2)], 1)
    table[0, 1:] = torch.cat([free[:2], free[4:5]])
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0, 0]), i32(lens), table, st)
    k, v = keys_values(gen, 70, 2, 64)
    for i in range(35):
        for b in range(2):
            at = slots_of(table[b], [lens[b]], 32) if lens[b] < 128 else torch.tensor([-1], device=DEV)
            lw.lw_kv_write(cache, k[2 * i + b:2 * i + b + 1], v[2 * i + b:2 * i + b + 1], at, st)
        old = list(lens)
        lens = [n + 1 for n in lens]
        lw.lw_kv_summarise(cache, summary, i32(old), i32(lens), table, st)
    for b, n in enumerate(lens):
        want = summary_of(cache, table[b], n)
        got = fields(cache, summary, table[b, :-(-n // 32)])
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    before = summary.clone()     # nothing new: nothing written
    lw.lw_kv_summarise(cache, summary, i32(lens), i32(lens), table, st)
    assert torch.equal(summary, before) and int(st) == 0


def test_equal_pages_and_special_keys():
    """The same keys in every page: the lower pages win.  A page with a NaN key scores highest."""
    gen, st = generator(3), status()
    page, n = 16, 160
    cache, table, _ = filled(gen, [n], 1, 64, page)
    k, v = keys_values(gen, page, 1, 64)
    lw.lw_kv_write(cache, k.repeat(10, 1, 1), v.repeat(10, 1, 1), slots_of(table[0], range(n), page), st)
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0]), i32([n]), table, st)
    q = torch.randn(1, 2, 64, device=DEV, generator=gen)
    got = attend(cache, summary, q, [0, 1], [n], table, st, 5, 1, 1)
    assert got[2].tolist() == [[[0, 1, 2, 3, 9]]]
    check(cache, q, [0, 1], [n], table, 5, 1, 1, 0.125, got, TOL["fp32"])
    k[0] = math.nan
    lw.lw_kv_write(cache, k[:1], v[:1], slots_of(table[0], [7 * page + 3], page), st)
    lw.lw_kv_summarise(cache, summary, i32([7 * page + 3]), i32([7 * page + 4]), table, st)
    lw.lw_kv_summarise(cache, summary, i32([0]), i32([n]), table, st)
    got = attend(cache, summary, q, [0, 1], [n], table, st, 5, 1, 1)
    assert got[2].tolist() == [[[0, 1, 2, 7, 9]]] and bool(torch.isnan(got[0]).all())
    # queries of nothing, and ones that are not finite: every score is 0
    for bad in (0.0, math.nan, math.inf, 1e-35):
        q[:] = bad
        lw.lw_kv_write(cache, v[:1] * 0 + 1, v[:1], slots_of(table[0], [7 * page + 3], page), st)
        lw.lw_kv_summarise(cache, summary, i32([0]), i32([n]), table, st)
        assert attend(cache, summary, q, [0, 1], [n], table, st, 5, 1, 1)[2].tolist() == [[[0, 1, 2, 3, 9]]]
    # keys of nothing
    k.zero_()
    lw.lw_kv_write(cache, k.repeat(10, 1, 1), v.repeat(10, 1, 1), slots_of(table[0], range(n), page), st)
    lw.lw_kv_summarise(cache, summary, i32([0]), i32([n]), table, st)
    q.fill_(1.0)
    assert attend(cache, summary, q, [0, 1], [n], table, st, 5, 1, 1)[2].tolist() == [[[0, 1, 2, 3, 9]]]
    assert int(st) == 0


def test_all_pages_is_attention():
    gen, st = generator(4), status()
    for typ in ("fp32", "bf16"):
        lens, start = [500, 70], [0, 3, 4]
        cache, table, _ = filled(gen, lens, 2, 128, 16)
        q = torch.randn(4, 8, 128, device=DEV, generator=gen).to(TYPES[typ])
        summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
        lw.lw_kv_summarise(cache, summary, i32([0, 0]), i32(lens), table, st)
        out, lse, _ = attend(cache, summary, q, start, lens, table, st, table.shape[1], 0, 1)
        ws = torch.zeros(lw.lw_kv_workspace_bytes(cache, 8, 4, 2), dtype=torch.uint8, device=DEV)
        full, flse = torch.empty_like(q), torch.empty(4, 8, device=DEV)
        lw.lw_kv_attention(cache, q, i32(start), i32(lens), table, full, ws, st, max_q=3, lse=flse)
        assert relative(out, full) <= 2 * TOL[typ] and float((lse - flse).abs().max()) < 1e-2
    assert int(st) == 0


def test_tokens_of_no_sequence_and_pages_that_are_not_there():
    gen, st = generator(5), status()
    lens, page = [200, 300], 16
    cache, table, _ = filled(gen, lens, 2, 64, page)
    q = torch.randn(6, 4, 64, device=DEV, generator=gen)
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0, 0]), i32(lens), table, st)
    start = [1, 3, 4]                     # rows 0, 4 and 5 belong to nobody
    got = attend(cache, summary, q, start, lens, table, st, 4, 1, 1)
    check(cache, q, start, lens, table, 4, 1, 1, 0.125, got, TOL["fp32"])
    for x, left in zip(got, (5, 5, -9)):
        assert bool((x[[0, 4, 5]] == left).all())
    assert int(st) == 0
    out = attend(cache, summary, q, [0, 9, 4], lens, table, st, 4, 1, 1)[0]      # not a range
    assert int(st) == lw.LW_DEV_BAD_SEQ and bool((out == 5).all())
    st, bad = status(), table.clone()
    bad[0, 12] = -1                       # the newest page of the first sequence, always read
    attend(cache, summary, q, start, lens, bad, st, 4, 1, 1)
    assert int(st) == lw.LW_DEV_BAD_PAGE
    st = status()
    lw.lw_kv_summarise(cache, summary, i32([0, 0]), i32(lens), bad, st)
    assert int(st) == lw.LW_DEV_BAD_PAGE
    st = status()
    attend(cache, summary, q, start, [200, 5000], table, st, 4, 1, 1)
    assert int(st) == lw.LW_DEV_BAD_SEQ


def test_replayed():
    gen, st = generator(6), status()
    lens, start, page = [900, 300], [0, 1, 2], 32
    cache, table, _ = filled(gen, lens, 2, 128, page)
    q = torch.randn(2, 8, 128, device=DEV, generator=gen).to(torch.bfloat16)
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    ws = torch.zeros(lw.lw_kv_blocks_workspace_bytes(cache, 8, 2, table.shape[1], 6), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(2, 8, device=DEV)
    chosen = torch.empty(2, 2, 6, dtype=torch.int32, device=DEV)
    qs, zero, n = i32(start), i32([0, 0]), i32(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = lw.StepGraph(side)
    with g.capture():
        lw.lw_kv_summarise(cache, summary, zero, n, table, st)
        lw.lw_kv_attention_blocks(cache, summary, q, qs, n, table, out, ws, st, blocks=6, first=1, recent=2, lse=lse,
                                  chosen=chosen)
    for now in ([900, 300], [640, 33], [899, 1]):
        q.copy_(torch.randn(2, 8, 128, device=DEV, generator=gen))
        n.copy_(i32(now))
        torch.cuda.synchronize()
        g.launch()
        torch.cuda.synchronize()
        check(cache, q, start, now, table, 6, 1, 2, 1 / math.sqrt(128), (out, lse, chosen), TOL["bf16"])
    assert int(st) == 0


@pytest.mark.parametrize("batch", [1, 120])
def test_thousands_of_pages(batch):
    """6250 pages of 16 keys: shared by a cluster, or (many heads of sequences) one CTA's."""
    gen, st, n, page = generator(7), status(), 100000, 16
    cache, table, _ = filled(gen, [n], 2, 64, page)
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0]), i32([n]), table, st)
    q = torch.randn(batch, 4, 64, device=DEV, generator=gen)
    # sequences that share their pages: queries at any position
    lens = [n - 800 * i for i in range(batch)]
    got = attend(cache, summary, q, list(range(batch + 1)), lens, table.expand(batch, -1).contiguous(), st, 70, 2, 3)
    assert int(st) == 0
    chi, clo, step = summary_of(cache, table[0], n)
    for b in range(0, batch, 17):
        # (the last page of a shorter sequence is summed up whole, and always read)
        nb = (lens[b] - 1) // page + 1
        for h in range(2):
            c, u = coded(q[b, 2 * h:2 * h + 2], q[b, 2 * h:2 * h + 2].abs().amax(-1, keepdim=True))
            dot = torch.maximum(c[:, None] * chi[:nb, h], c[:, None] * clo[:nb, h]).double().sum(-1).float()
            score = (dot * u).amax(0) * step[:nb, h]
            assert got[2][b, h].tolist() == chosen_by(score.tolist(), nb, 70, 2, 3)
    check(cache, q[:1], [0, 1], lens[:1], table, 70, 2, 3, 0.125, [x[:1] for x in got], TOL["fp32"])


WIDTHS = """
import sys
import torch
from decode_gemv_gb300 import lw

def run(group, widths):
    heads, dim, page, blocks = 8, 128, 16, 3
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tokens = 6 * sms // (2 * heads) + 2                 # too many tokens and heads for clusters: one CTA has a table
    cache = lw.KvCache.empty(4, heads, dim, page, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    cache.pages.zero_()
    st, start = torch.zeros(1, **i32), torch.arange(tokens + 1, **i32)
    n, q = torch.full((tokens,), 64, **i32), torch.ones(tokens, heads * group, dim, device="cuda")
    summary, out = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    chosen = torch.empty(tokens, heads, blocks, **i32)
    for width in widths:
        table = torch.full((tokens, width), -1, **i32)
        table[:, :4] = torch.arange(4, **i32)
        need = lw.lw_kv_blocks_workspace_bytes(cache, heads * group, tokens, width, blocks)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        lw.lw_kv_attention_blocks(cache, summary, q, start, n, table, out, ws, st, blocks=blocks, chosen=chosen)
        assert bool((chosen == torch.tensor([0, 1, 3], **i32)).all()) and int(st) == 0, (group, width)

for group in (4, 1, 16):
    # around 48 KB of order keys, heads' codes and the choice's own, and up to the widest
    room = (49152 - 4300 - 260 * group) // 4 - 32
    run(group, [*range(room - 24, room + 12, 4), 20000, 40960])
print("done")
"""


def test_any_width_of_the_page_table():
    """In a process of its own: what a kernel may take of shared memory is raised by wider tables and stays so."""
    import subprocess
    import sys
    from pathlib import Path
    r = subprocess.run([sys.executable, "-c", WIDTHS], capture_output=True, text=True, timeout=300,
                       cwd=Path(__file__).resolve().parent.parent)
    assert r.returncode == 0 and r.stdout.split()[-1] == "done", r.stdout + r.stderr


@pytest.mark.parametrize("case", [(8, 1, 128, 64), (16, 16, 64, 16), (6, 2, 96, 48)], ids=str)
def test_bf16_operands_hold_their_bits(case):
    """Before the output's rounding a bf16 call is within 2^-11, as lw_kv_attention's few rows are (probabilities, and
    these times the values' scales, in 11 bits each: 2^-12 at most).  The rounding's own error is known from the exact
    result; independent errors add as squares (2 % for chance).  So a call may differ from one that carries 32 bits
    throughout by as many outputs as lie that near the middle between two bf16 numbers."""
    hq, h, dim, page = case
    gen, st, lens = generator(60), status(), [3000, 2500, 2000, 1000]
    cache, table, _ = filled(gen, lens, h, dim, page)
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0] * 4), i32(lens), table, st)
    q = torch.randn(8, hq, dim, device=DEV, generator=gen).to(torch.bfloat16)
    out, _, chosen = attend(cache, summary, q, [0, 2, 4, 6, 8], lens, table, st, 640 // page, 1, 2)
    want = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for i in range(8):
        n = lens[i // 2]
        k, v = (x.double() for x in read(cache, slots_of(table[i // 2], range(n), page)))
        for g in range(h):
            rows = slice(g * (hq // h), (g + 1) * (hq // h))
            at = [x for x in chosen[i, g].tolist() if x >= 0]
            pos = n - 2 + i % 2
            key = torch.tensor([j for x in at for j in range(x * page, min(x * page + page, pos + 1))], device=DEV)
            want[i, rows] = (q[i, rows].double() @ k[key, g].T / math.sqrt(dim)).softmax(-1) @ v[key, g]
    r = relative(want.to(torch.bfloat16), want)
    assert int(st) == 0 and relative(out, want) <= 1.02 * math.hypot(r, 2.0 ** -11)


@pytest.mark.parametrize("case", [(4, 1, 128, 64), (2, 2, 64, 16), (8, 1, 96, 48)], ids=str)
def test_scores_stand_for_unrounded_ranges(case):
    """A page's score is its ranges' upper bound on q.k, sum max(q lo, q hi), but for 8-bit codes: each element is off
    by at most half a step, so the sum by E = sum |q| step / 2 + |k| u / 2 + step u / 4 (1e-4 of it for fp32 steps: a
    code's quotient is near 127 to 2^-22).  No page that was left out has an unrounded score above a chosen one's by
    more than their two E."""
    hq, h, dim, page = case
    gen, st, n, blocks, first, recent = generator(61), status(), 6000, 20, 1, 2
    cache, table, _ = filled(gen, [n], h, dim, page)
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0]), i32([n]), table, st)
    q = torch.randn(6, hq, dim, device=DEV, generator=gen)
    _, _, chosen = attend(cache, summary, q, [0, 6], [n], table, st, blocks, first, recent)
    assert int(st) == 0
    k, nb = read(cache, slots_of(table[0], range(n), page))[0].double(), -(-n // page)
    k = torch.cat([k, k[-1:].expand(nb * page - n, h, dim)]).view(nb, page, h, dim)
    lo, hi = k.amin(1), k.amax(1)
    size = torch.maximum(lo.abs(), hi.abs())
    step = size.amax(-1, keepdim=True) / 127
    for i in range(6):
        pages = (n - 6 + i) // page + 1
        for g in range(h):
            rows = q[i, g * (hq // h):(g + 1) * (hq // h)].double()[:, None]       # [group, 1, dim]
            u = rows.abs().amax(-1, keepdim=True) / 127
            true = torch.maximum(rows * lo[:pages, g], rows * hi[:pages, g]).sum(-1)
            off = (rows.abs() * step[:pages, g] / 2 + size[:pages, g] * u / 2 + step[:pages, g] * u / 4).sum(-1)
            score, off = true.amax(0), off.amax(0) * (1 + 1e-4) + 1e-5 * true.abs().amax(0)
            took = torch.zeros(pages, dtype=torch.bool, device=DEV)
            took[chosen[i, g].long()] = True
            free = torch.ones_like(took)
            free[:first], free[pages - recent:] = False, False
            ins, outs = took & free, ~took & free
            assert int(ins.sum()) == blocks - first - recent
            assert float((score + off)[ins].min()) >= float((score - off)[outs].max())
