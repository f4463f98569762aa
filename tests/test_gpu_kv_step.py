"""The calls around the 4-bit cache as a generator uses them together: prompts written with rotary positions,
attention and its weights, eviction in place, then decode steps (rotary write, summaries, block-sparse attention,
full attention with its weights added up) captured once and replayed.  Each result against 64 bits on the cached
values of the same moment, with the tolerances of the calls' own tests."""
import math

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from kv_plain import DEV, generator, i32, pool, read, relative, scores, slots_of, spans, status
HQ, H, D, PAGE, KEEP, FIRST, RECENT, BLOCKS = 8, 2, 128, 16, 128, 4, 32, 5
LENS, STEPS = [300, 90], 40


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def rotated(x, row):
    c, s = row[:, None, :D // 2], row[:, None, D // 2:]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_generation(typ):
    tol = 1e-4 if typ == torch.float32 else 1.5e-2
    gen, st, batch, total = generator(77), status(), len(LENS), sum(LENS)
    width = -(-max(LENS) // PAGE) + 4
    cache = pool(gen, batch * width, H, D, PAGE)
    table = torch.randperm(batch * width, device=DEV, generator=gen).to(torch.int32).view(batch, width)
    angles = torch.empty(1000, D, device=DEV)
    lw.lw_rotary_table(angles, base=500000.0, scaling=lw.LW_ROTARY_BANDS, factor=8.0, old_length=256.0)
    keys = width * PAGE
    weights = torch.zeros(batch, H, keys, device=DEV)
    scale = 1 / math.sqrt(D)

    # ---- the prompts: one product's output, queries rotated in place
    qkv = torch.randn(total, HQ + 2 * H, D, device=DEV, generator=gen).to(typ)
    before = qkv.float().clone()     # (the rotation is in place)
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:]
    pos = torch.cat([torch.arange(n, device=DEV) for n in LENS])
    slots = torch.cat([slots_of(table[b], range(n), PAGE) for b, n in enumerate(LENS)])
    lw.lw_kv_write_rotary(cache, k, v, slots, pos, angles, st, q=q, q_out=q)
    assert torch.equal(q, rotated(before[:, :HQ], angles[pos]).to(typ))
    start = [0, LENS[0], total]
    out, lse = torch.empty(total, HQ, D, dtype=typ, device=DEV), torch.empty(total, HQ, device=DEV)
    ws = torch.zeros(lw.lw_kv_workspace_bytes(cache, HQ, total, batch), dtype=torch.uint8, device=DEV)
    lw.lw_kv_attention(cache, q, i32(start), i32(LENS), table, out, ws, st, max_q=max(LENS), lse=lse)
    wws = torch.empty(lw.lw_kv_weigh_workspace_bytes(cache, HQ, total), dtype=torch.uint8, device=DEV)
    lw.lw_kv_weigh(cache, q, lse, i32(start), i32(LENS), table, weights, wws, st, max_q=max(LENS))
    for b, n in enumerate(LENS):
        kk, vv = read(cache, slots_of(table[b], range(n), PAGE))
        s = scores(q[start[b]:start[b + 1]], kk, spans(n, n), scale)
        want = s.softmax(-1)
        assert relative(weights[b, :, :n], want.view(n, H, HQ // H, n).sum((0, 2))) <= tol
        o = torch.einsum("thj,jhd->thd", want, vv.double().repeat_interleave(HQ // H, 1))
        assert relative(out[start[b]:start[b + 1]], o) <= tol

    # ---- eviction in place
    before_w, before_kv = weights.clone(), [read(cache, slots_of(table[b], range(n), PAGE)) for b, n in enumerate(LENS)]
    kept, lens = torch.empty(batch, H, KEEP, dtype=torch.int32, device=DEV), i32([0] * batch)
    lw.lw_kv_evict(cache, weights, i32(LENS), table, table, lens, weights, kept, st, keep=KEEP, first=FIRST,
                   recent=RECENT)
    assert lens.tolist() == [min(n, KEEP) for n in LENS]
    for b, n in enumerate(LENS):
        m = min(n, KEEP)
        now = read(cache, slots_of(table[b], range(m), PAGE))
        for h in range(H):
            at = kept[b, h, :m].long()
            assert torch.equal(weights[b, h, :m], before_w[b, h, at]) and not bool(weights[b, h, m:].any())
            assert all(torch.equal(x[:, h], y[at, h]) for x, y in zip(now, before_kv[b]))
            if n > KEEP:
                rest = sorted(range(FIRST, n - RECENT), key=lambda j: (-float(before_w[b, h, j]), j))
                assert sorted(at.tolist()) == sorted([*range(FIRST), *range(n - RECENT, n),
                                                      *rest[:KEEP - FIRST - RECENT]])
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0] * batch), lens, table, st)

    # ---- a decode step, captured once; what changes lies in buffers
    step = torch.empty(batch, HQ + 2 * H, D, dtype=typ, device=DEV)
    q, k, v = step[:, :HQ], step[:, HQ:HQ + H], step[:, HQ + H:]
    slot, at = torch.empty(batch, dtype=torch.int64, device=DEV), torch.empty(batch, dtype=torch.int64, device=DEV)
    old, qs = lens.clone(), i32(list(range(batch + 1)))
    sparse, full = (torch.empty(batch, HQ, D, dtype=typ, device=DEV) for _ in range(2))
    lse, chosen = torch.empty(batch, HQ, device=DEV), torch.empty(batch, H, BLOCKS, dtype=torch.int32, device=DEV)
    bws = torch.zeros(lw.lw_kv_blocks_workspace_bytes(cache, HQ, batch, width, BLOCKS), dtype=torch.uint8, device=DEV)
    aws = torch.zeros(lw.lw_kv_workspace_bytes(cache, HQ, batch, batch), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = lw.StepGraph(side)
    with g.capture():
        lw.lw_kv_write_rotary(cache, k, v, slot, at, angles, st, q=q, q_out=q)
        lw.lw_kv_summarise(cache, summary, old, lens, table, st)
        lw.lw_kv_attention_blocks(cache, summary, q, qs, lens, table, sparse, bws, st, blocks=BLOCKS, first=1,
                                  recent=2, chosen=chosen)
        lw.lw_kv_attention(cache, q, qs, lens, table, full, aws, st, max_q=1, lse=lse)
        lw.lw_kv_weigh(cache, q, lse, qs, lens, table, weights, wws, st, max_q=1, add_to=weights)
    for i in range(STEPS):
        step.copy_(torch.randn(step.shape, device=DEV, generator=gen))
        old.copy_(lens)
        slot.copy_(torch.stack([table[b].long()[int(n) // PAGE] * PAGE + int(n) % PAGE for b, n in enumerate(lens)]))
        at.copy_(torch.tensor([n + i for n in LENS]))
        lens += 1
        had = weights.clone()
        torch.cuda.synchronize()
        g.launch()
        torch.cuda.synchronize()
        if i % 13:
            continue
        for b, n in enumerate(lens.tolist()):
            kk, vv = (x.double() for x in read(cache, slots_of(table[b], range(n), PAGE)))
            s = scores(q[b:b + 1], kk, spans(1, n), scale)[0]
            o = torch.einsum("hj,jhd->hd", s.softmax(-1), vv.repeat_interleave(HQ // H, 1))
            assert relative(full[b], o) <= tol
            w = s.softmax(-1).view(H, HQ // H, n).sum(1)
            assert relative(weights[b, :, :n] - had[b, :, :n], w) <= tol
            nb = (n - 1) // PAGE + 1
            for h in range(H):
                pages = [x for x in chosen[b, h].tolist() if x >= 0]
                assert len(pages) == min(nb, BLOCKS) and pages[0] == 0 and pages[-2:] == [nb - 2, nb - 1]
                key = torch.tensor([j for x in pages for j in range(x * PAGE, min(x * PAGE + PAGE, n))], device=DEV)
                heads = slice(h * (HQ // H), (h + 1) * (HQ // H))
                assert relative(sparse[b, heads], s[heads][:, key].softmax(-1) @ vv[key, h]) <= tol
    assert int(st) == 0


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_one_workspace_for_all_calls(typ):
    """A workspace of the largest size, zeroed once, serves attention, its weights and sparse attention in turn: the
    same bits as with workspaces of their own.  (Items are cut between CTAs here, which the counters in front join.)"""
    gen, st, n = generator(78), status(), 5000
    cache = pool(gen, 320, H, D, PAGE)
    table = torch.randperm(320, device=DEV, generator=gen).to(torch.int32).view(1, 320)
    kv = torch.randn(2, n, H, D, device=DEV, generator=gen)
    lw.lw_kv_write(cache, kv[0], kv[1], slots_of(table[0], range(n), PAGE), st)
    summary = torch.zeros(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0]), i32([n]), table, st)

    def sizes(tokens):
        return (lw.lw_kv_workspace_bytes(cache, HQ, tokens, 1), lw.lw_kv_weigh_workspace_bytes(cache, HQ, tokens),
                lw.lw_kv_blocks_workspace_bytes(cache, HQ, tokens, 320, 200))

    def zeros(size):
        return torch.zeros(max(size, 16), dtype=torch.uint8, device=DEV)

    def step(q, tokens, attn, weigh, blocks):
        out, sparse, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(tokens, HQ, device=DEV)
        w = torch.empty(1, H, n, device=DEV)
        args = (i32([0, tokens]), i32([n]), table)
        lw.lw_kv_attention(cache, q, *args, out, attn, st, max_q=tokens, lse=lse)
        lw.lw_kv_weigh(cache, q, lse, *args, w, weigh, st, max_q=tokens)
        lw.lw_kv_attention_blocks(cache, summary, q, *args, sparse, blocks, st, blocks=200)
        return out, lse, w, sparse

    ws = zeros(max(max(sizes(t)) for t in (1, 7, 300)))
    for tokens in (300, 1, 7, 300, 1):
        q = torch.randn(tokens, HQ, D, device=DEV, generator=gen).to(typ)
        want = step(q, tokens, *(zeros(x) for x in sizes(tokens)))
        got = step(q, tokens, ws, ws, ws)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), tokens
    assert int(st) == 0
