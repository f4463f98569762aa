"""Operators around the 4-bit key/value cache: what they compute, at the sizes they are used at.

A token generator that keeps its keys and values in 4 bits needs, next to the
write, the read-back and the attention,

* rotary positions (lw_kv_write_rotary): the tokens' queries and keys are
  rotated by their positions' angles as the keys and values are stored;
* eviction by accumulated attention weight: the softmax weights that each
  cached key was given, summed over the queries (lw_kv_weigh), and the cache cut
  down to the first, the newest and the heaviest keys of each head (lw_kv_evict);
* sparse attention over blocks (lw_kv_summarise, lw_kv_attention_blocks): a
  page's keys are summed up by their channelwise range in 8 bits, a query is
  scored against the ranges, and attends to the pages that score highest.

Layout of the cache.  A page holds `page` token slots (a multiple of 16) for
every key/value head: [kv_heads][page / 16] tiles of 16 tokens.  A tile, in
16-bit units, with G = D / 32 groups and GP = G rounded up to an even number:
  key codes      ((t * 4 + q) * G + g) * 2 + h, nibble i: d = 32 g + 8 q + 4 h + i
  key scales     [t / 2][g][t % 2]    fp16
  key minimums   [t][GP]              fp16
  value codes    (((t / 2) * 8 + n) * G + g) * 2 + t % 2, nibble i: d = 32 g + 4 n + i
  value scales   [t / 2][g][t % 2]    fp16
  value minimums [t / 2][g][t % 2]    fp16
A sequence's tokens lie in the pages its row of the page table names.
"""
import math
import random

import torch

own = False

GROUP = 32
LIMIT = 61440.0   # larger magnitudes are held as this one (15 scale + minimum stays in fp16)
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one decode step of one sequence, far into a long context: the fp32 outputs of the
        # coded q, k and v products
        dict(name="rotary 1 token fp32", op="rotary", tokens=1, q_heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, scaling="bands", page=64, type="fp32", skip=0,
             positions=131072),
        # one decode step of a padded batch: half of the head is rotated, in neighbouring pairs
        dict(name="rotary 61 tokens fp32", op="rotary", tokens=61, q_heads=32, kv_heads=32, dim=96,
             rot=48, interleaved=True, scaling="none", page=16, type="fp32", skip=5,
             positions=4096),
        # a long prompt
        dict(name="rotary 65536 tokens bf16", op="rotary", tokens=65536, q_heads=32, kv_heads=8,
             dim=128, rot=128, interleaved=False, scaling="yarn", page=64, type="bf16", skip=0,
             positions=65536),
        # the weights that one decode step of one sequence gives
        dict(name="weigh 1x4097 fp32", op="weigh", batch=1, q_heads=32, kv_heads=8, dim=128,
             page=64, type="fp32", q_min=1, q_max=1, len_min=4097, len_max=4097, window=0,
             causal=True, add=True, past=False, shape=1),
        # one decode step of few sequences with very long contexts
        dict(name="weigh 8 long bf16", op="weigh", batch=8, q_heads=32, kv_heads=8, dim=128,
             page=256, type="bf16", q_min=1, q_max=1, len_min=20000, len_max=131072, window=0,
             causal=True, add=True, past=False, shape=2),
        # a chunk of a long prompt
        dict(name="weigh 2048 on 14336 bf16", op="weigh", batch=1, q_heads=32, kv_heads=8, dim=128,
             page=64, type="bf16", q_min=2048, q_max=2048, len_min=14336, len_max=14336, window=0,
             causal=True, add=False, past=True, shape=3),
        # one sequence cut in half
        dict(name="evict 1x4500", op="evict", batch=1, kv_heads=8, dim=128, page=64,
             len_min=4500, len_max=4500, keep=2250, first=4, recent=256, shape=4),
        # a served batch, not all of it over its limit
        dict(name="evict 16 ragged", op="evict", batch=16, kv_heads=8, dim=128, page=64,
             len_min=0, len_max=9000, keep=2048, first=4, recent=128, shape=5),
        # long contexts cut to an eighth
        dict(name="evict 8x65536", op="evict", batch=8, kv_heads=8, dim=128, page=256,
             len_min=65536, len_max=65536, keep=8192, first=4, recent=1024, shape=6),
        # one decode step in the middle of an answer
        dict(name="blocks 1x4097 fp32", op="blocks", batch=1, q_heads=32, kv_heads=8, dim=128,
             page=64, type="fp32", q_max=1, len_min=4097, len_max=4097, fresh=1, blocks=16,
             first=1, recent=2, shape=7),
        # five drafted tokens of each of 16 sequences, small pages, a head of keys for every head
        # of queries
        dict(name="blocks 16x5 fp16", op="blocks", batch=16, q_heads=16, kv_heads=16, dim=64,
             page=16, type="fp16", q_max=5, len_min=1000, len_max=9000, fresh=5, blocks=48,
             first=1, recent=4, shape=8),
        # the first step after very long prompts: every page is summed up, 64 of up to 2048 are read
        dict(name="blocks 8 long bf16", op="blocks", batch=8, q_heads=32, kv_heads=8, dim=128,
             page=64, type="bf16", q_max=1, len_min=20000, len_max=131072, fresh=131072, blocks=64,
             first=1, recent=4, shape=9),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high))))))


def draw(rng):
    op = rng.choice(["rotary", "weigh", "weigh", "evict", "blocks"])
    dim = rng.choice([64, 96, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
    group = rng.choice([1, 1, 2, 4, 4, 8]) if kv_heads < 32 else 1
    page = rng.choice([16, 32, 48, 64, 128, 256])
    typ = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    case = dict(op=op, kv_heads=kv_heads, dim=dim, page=page)
    if op == "rotary":
        top = 65536 * 48 * 128 // ((kv_heads * (group + 2)) * dim * (2 if typ == "fp32" else 1))
        return dict(case, tokens=_log(rng, 1, min(65536, top)), q_heads=kv_heads * group, type=typ,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)]),
                    interleaved=rng.random() < 0.5, skip=rng.choice([0, 0, 7]),
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                    positions=_log(rng, 1000, 200000))
    case.update(shape=rng.randrange(1 << 20), batch=_log(rng, 1, 100))
    room = min(131072, (1 << 29) // (case["batch"] * kv_heads * dim))   # cached tokens a sequence
    if op == "evict":
        top = _log(rng, 1, room)
        case.update(len_max=top, len_min=rng.choice([0, 1, top // 2, top]),
                    keep=_log(rng, 1, max(2, top)))
        case["recent"] = rng.randint(0, case["keep"])
        case["first"] = min(rng.choice([0, 1, 4, 33]), case["keep"] - case["recent"])
        return case
    case.update(q_heads=kv_heads * group, type=typ)
    if op == "blocks":
        case["q_max"] = rng.choice([1, 1, 1, 2, 5, 8])
        if kv_heads * case["q_max"] * case["batch"] > 16384:
            case["q_max"] = 1
        blocks = _log(rng, 2, 96)
        # what is read of each query's keys stays within the listed ones
        rows = kv_heads * case["q_max"] * case["batch"]
        blocks = max(2, min(blocks, (1 << 26) // (rows * page * dim)))
        top = max(2, min(_log(rng, 1, room), page * 40000))
        case.update(blocks=blocks, recent=rng.randint(1, max(1, blocks // 4)), len_max=top,
                    len_min=rng.choice([1, top // 2, top]),
                    fresh=rng.choice([case["q_max"], case["q_max"], 300, 131072]))
        case["first"] = min(rng.choice([0, 1, 2]), blocks - case["recent"])
        return case
    chunk = rng.random() < 0.4
    case.update(q_min=1, q_max=1, window=rng.choice([0, 0, 0, 129, 4096]), causal=True,
                add=rng.random() < 0.5, past=chunk, len_min=0, len_max=0)
    if chunk:
        case["q_max"] = _log(rng, 9, 4096)
        case["q_min"] = rng.choice([0, case["q_max"] // 2, case["q_max"]])
        case["batch"] = _log(rng, 1, 6)
        top = min(32768, (1 << 29) // (case["batch"] * case["q_heads"] * case["q_max"]))
        past = max(0, top - case["q_max"])
        case["len_max"] = _log(rng, 1, past) if past > 1 else 0
        case["len_min"] = rng.choice([0, case["len_max"] // 2, case["len_max"]])
    else:
        case["q_max"] = rng.choice([1, 1, 1, 2, 4, 7])
        case["len_max"] = max(1, _log(rng, 1, max(2, room // case["q_max"])))
        case["len_min"] = rng.choice([0, 1, case["len_max"] // 8, case["len_max"]])
        case["causal"] = rng.random() < 0.8
    return case


def _lengths(case):
    """Query tokens and cached keys (the new tokens' own among them) of each sequence."""
    rng = random.Random(case["shape"])
    q, kv = [], []
    for _ in range(case["batch"]):
        t = rng.randint(case.get("q_min", 1), case.get("q_max", 1))
        n = rng.randint(case["len_min"], case["len_max"])
        q.append(t)
        # a chunk comes on top of what is cached; a decode step's length counts its own tokens
        kv.append(n + t if case.get("past") else max(n, t) if case["op"] == "blocks" else n)
    q[0], kv[0] = max(q[0], 1), max(kv[0], 1)
    return q, kv


def _tile_units(dim):
    """16-bit units of the six parts of a tile of 16 tokens."""
    g = dim // GROUP
    return [4 * dim, 16 * g, 16 * (g + g % 2), 4 * dim, 16 * g, 16 * g]


def _size(case):
    return 4 if case["type"] == "fp32" else 2


def work(case):
    """Inputs once, outputs once; of the cache the codes, scales and minimums of the keys (and
    values) that the call has to see or to write."""
    d, h = case["dim"], case["kv_heads"]
    half = d // 2 + 4 * (d // GROUP)   # cached bytes of one token's key head, or value head
    if case["op"] == "rotary":
        n, hq, size = case["tokens"], case["q_heads"], _size(case)
        kept = n - (n // case["skip"] if case["skip"] else 0)
        # queries in and out, keys and values in and (read back) out, the cache written and read
        return {"bytes": kept * (2 * hq * d * size + 4 * h * d * size + 4 * h * half + 4 * case["rot"])
                + 16 * n, "flops": kept * (3.0 * (hq + h) * case["rot"] + 16.0 * h * d)}
    q_len, kv_len = _lengths(case)
    if case["op"] == "evict":
        byts = 0
        for n in kv_len:
            m = min(n, case["keep"])
            # weights in; kept tokens in and out, and (read back) out as 16-bit values
            byts += h * (4 * n + 8 * m + m * (6 * half + 4 * d))
        return {"bytes": byts, "flops": float(h * sum(kv_len))}
    size, hq = _size(case), case["q_heads"]
    byts, flops = 0, 0.0
    for t, n in zip(q_len, kv_len):
        if case["op"] == "weigh":
            first = max(0, n - t - case["window"] + 1) if case["window"] else 0
            byts += t * hq * (d * size + 4) + h * (n - first) * half + h * n * (8 if case["add"] else 4)
            flops += 2.0 * hq * d * sum(hi - lo for lo, hi in _spans(case, t, n))
        else:
            nb = -(-n // case["page"])
            new = min(nb, -(-min(case["fresh"], n) // case["page"]))
            # the new pages' keys, the summaries, and each query's pages a head
            byts += 2 * t * hq * d * size + h * (min(n, new * case["page"]) * half + (nb + new) * (2 * d + 4))
            byts += t * h * min(n, case["blocks"] * case["page"]) * 2 * half
            flops += t * hq * d * (4.0 * nb + 4.0 * min(n, case["blocks"] * case["page"]))
    return {"bytes": byts, "flops": flops}


def _spans(case, t, n):
    """[lo, hi) of the keys each of t tokens may see."""
    out = []
    for i in range(t):
        pos = n - t + i
        hi = max(0, min(n, pos + 1)) if case["causal"] else n
        lo = max(0, pos - case["window"] + 1) if case["window"] else 0
        out.append((min(lo, hi), hi))
    return out


# ----------------------------------------------------------------------------
# what a program has in hand before the call
# ----------------------------------------------------------------------------

def _keys_values(gen, n, heads, dim):
    """Keys and values as a layer makes them: unit spread, with a few key channels of a head
    that are large and have an offset."""
    k = torch.randn(n, heads, dim, device=DEV, generator=gen)
    v = torch.randn(n, heads, dim, device=DEV, generator=gen)
    gain = 1 + 3 * (torch.rand(heads, dim, device=DEV, generator=gen) < 0.03)
    shift = 2 * torch.randn(heads, dim, device=DEV, generator=gen) * (gain > 1)
    return k * gain + shift, v


def _page_shape(case, pages):
    return (pages, case["kv_heads"], case["page"] // 16, sum(_tile_units(case["dim"])))


def _stale(gen, shape):
    """Pages as memory has them before they are written: any bits."""
    words = math.prod(shape)
    return torch.randint(0, 256, (words * 2,), dtype=torch.uint8, device=DEV,
                         generator=gen).view(torch.int16).view(shape)


def _frequencies(case):
    """Angle per position of each pair, and the factor on cosines and sines (fp64)."""
    base, factor, old = 10000.0, 8.0, 8192.0
    rot, kind = case["rot"], case["scaling"]
    if kind == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    f = base ** (-2 * i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "bands":      # long waves are stretched, short ones kept, those between blended
        turns = old * f / (2 * math.pi)
        keep = ((turns - 1) / 3).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 1.0
    if kind == "yarn":
        def pair(rounds):    # the pair that makes so many turns in the old length
            return rot * math.log(old / (rounds * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(0, math.floor(pair(32.0))), min(rot - 1, math.ceil(pair(1.0)))
        keep = 1 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1
    return f, 1.0


def _table(case):
    """[positions, rot] fp32: the pairs' cosines, then their sines."""
    f, m = _frequencies(case)
    a = torch.arange(case["positions"], device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([torch.cos(a) * m, torch.sin(a) * m], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    state = {"rotary": _rotary_state, "weigh": _weigh_state, "evict": _evict_state,
             "blocks": _blocks_state}[case["op"]](case, gen)
    if own:   # the handle, workspace and status word that a user's program keeps
        from decode_gemv_gb300 import lw
        cache = lw.KvCache(state["pages"].view(torch.uint8), case["kv_heads"], case["dim"], case["page"])
        state["cache"], state["status"] = cache, torch.zeros(1, dtype=torch.int32, device=DEV)
        need = 0
        if case["op"] == "weigh":
            need = lw.lw_kv_weigh_workspace_bytes(cache, case["q_heads"], state["q"].shape[0])
        elif case["op"] == "blocks":
            need = lw.lw_kv_blocks_workspace_bytes(cache, case["q_heads"], state["q"].shape[0],
                                                   state["table"].shape[1], case["blocks"])
        state["ws"] = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    return state


def _rotary_state(case, gen):
    n, page, typ = case["tokens"], case["page"], TYPES[case["type"]]
    k, v = _keys_values(gen, n, case["kv_heads"], case["dim"])
    q = 1.5 * torch.randn(n, case["q_heads"], case["dim"], device=DEV, generator=gen)
    pages = -(-n // page) + 1
    # runs of 16 slots in any order, as pages are handed out
    runs = torch.randperm((pages - 1) * (page // 16), device=DEV, generator=gen)
    slots = (runs[:, None] * 16 + torch.arange(16, device=DEV)).reshape(-1)[:n].contiguous()
    # consecutive positions up to the newest one, round and round where there are more tokens
    last = case["positions"] - 1 - torch.randint(0, 50, (1,), device=DEV, generator=gen)
    pos = (last - n + 1 + torch.arange(n, device=DEV)) % case["positions"]
    if case["skip"]:
        slots[case["skip"] - 1::case["skip"]] = -1
        pos[case["skip"] - 1::case["skip"]] = -1
    return dict(case=case, q=q.to(typ), k=k.to(typ), v=v.to(typ), slots=slots, pos=pos,
                table=_table(case), q_out=torch.zeros(q.shape, dtype=typ, device=DEV),
                pages=_stale(gen, _page_shape(case, pages)))


def _sequences(case, gen, kv_len, spare=0):
    """Pages, written with keys and values, the page table, and the page ids left over."""
    page, batch = case["page"], case["batch"]
    used = [-(-n // page) for n in kv_len]
    width = max(max(used), 1)
    pages = sum(used) + 3 + spare
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)   # no page
    at = torch.tensor([0] + used, device=DEV).cumsum(0)
    col = torch.arange(width, device=DEV)
    has = col < torch.tensor(used, device=DEV)[:, None]
    table[has] = order[(at[:-1, None] + col)[has]]
    store = _stale(gen, _page_shape(case, pages))
    for b, n in enumerate(kv_len):   # sequence by sequence: the intermediates stay small
        if n:
            k, v = _keys_values(gen, n, case["kv_heads"], case["dim"])
            pos = torch.arange(n, device=DEV)
            _plain_write(store, case, k, v, table[b, pos // page].long() * page + pos % page)
    return store, table, order[sum(used) + 3:]


def _queries(case, gen, q_len):
    q = torch.randn(sum(q_len), case["q_heads"], case["dim"], device=DEV, generator=gen)
    start = torch.tensor([0] + q_len, device=DEV).cumsum(0).to(torch.int32)
    return (1.5 * q).to(TYPES[case["type"]]), start


def _weigh_state(case, gen):
    q_len, kv_len = _lengths(case)
    store, table, _ = _sequences(case, gen, kv_len)
    q, start = _queries(case, gen, q_len)
    width = max(kv_len)
    before = torch.rand(case["batch"], case["kv_heads"], width, device=DEV, generator=gen) ** 8
    s = dict(case=case, pages=store, q=q, q_start=start, table=table, max_q=max(q_len),
             kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV),
             before=before if case["add"] else None,
             weights=torch.zeros(case["batch"], case["kv_heads"], width, device=DEV))
    # the log-sums that attention over the same queries left
    s["lse"] = torch.full(q.shape[:2], -math.inf, device=DEV)
    group = case["q_heads"] // case["kv_heads"]
    for b, n in enumerate(kv_len):
        t, at = q_len[b], int(start[b])
        if t and n:
            k = _plain_keys(s, b).repeat_interleave(group, 0)
            x = q[at:at + t].float().transpose(0, 1) @ k[:, :n].transpose(1, 2) / math.sqrt(case["dim"])
            x.masked_fill_(~_visible(case, t, n), -math.inf)
            s["lse"][at:at + t] = x.logsumexp(-1).T
    return s


def _visible(case, t, n):
    pos = torch.arange(n - t, n, device=DEV)[:, None]
    key = torch.arange(n, device=DEV)[None]
    see = torch.ones(t, n, dtype=torch.bool, device=DEV)
    if case["causal"]:
        see &= key <= pos
    if case["window"]:
        see &= key > pos - case["window"]
    return see


def _evict_state(case, gen):
    _, kv_len = _lengths(case)
    page, batch, heads = case["page"], case["batch"], case["kv_heads"]
    to = -(-case["keep"] // page)
    store, table, free = _sequences(case, gen, kv_len, batch * to)
    width = max(kv_len)
    # sums of softmax weights: a few keys have most of it, many the same little or nothing
    w = torch.rand(batch, heads, width, device=DEV, generator=gen) ** 12
    w = torch.where(w < 1e-4, torch.floor(w * 2e5) * 5e-6, 30 * w)
    return dict(case=case, pages=store, table=table, weights=w,
                kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV),
                out_table=free.view(batch, to).contiguous(),
                out_len=torch.zeros(batch, dtype=torch.int32, device=DEV),
                out_weights=torch.zeros(batch, heads, case["keep"], device=DEV),
                kept=torch.zeros(batch, heads, case["keep"], dtype=torch.int32, device=DEV))


def _blocks_state(case, gen):
    q_len, kv_len = _lengths(case)
    store, table, _ = _sequences(case, gen, kv_len)
    q, start = _queries(case, gen, q_len)
    s = dict(case=case, pages=store, q=q, q_start=start, table=table, max_q=max(q_len),
             kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV),
             start=torch.tensor([max(0, n - case["fresh"]) for n in kv_len], dtype=torch.int32,
                                device=DEV),
             summary=torch.zeros(store.shape[0], case["kv_heads"], 2 * case["dim"] + 16,
                                 dtype=torch.uint8, device=DEV),
             out=torch.empty_like(q),
             chosen=torch.empty(q.shape[0], case["kv_heads"], case["blocks"], dtype=torch.int32,
                                device=DEV))
    # what earlier steps summed up
    _plain_summarise(s, torch.zeros_like(s["start"]), s["kv_len"], table.shape[1])
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    kind = state["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "weigh": _own_weigh, "evict": _own_evict,
                "blocks": _own_blocks}[kind](state)
    return {"rotary": _plain_rotary, "weigh": _plain_weigh, "evict": _plain_evict,
            "blocks": _plain_blocks}[kind](state)


def _own_rotary(s):
    from decode_gemv_gb300 import lw
    lw.lw_kv_write_rotary(s["cache"], s["k"], s["v"], s["slots"], s["pos"], s["table"], s["status"],
                          q=s["q"], q_out=s["q_out"], interleaved=s["case"]["interleaved"])
    k, v = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    lw.lw_kv_read(s["cache"], s["slots"], k, v, s["status"])
    return s["q_out"], k, v


def _own_weigh(s):
    from decode_gemv_gb300 import lw
    c = s["case"]
    lw.lw_kv_weigh(s["cache"], s["q"], s["lse"], s["q_start"], s["kv_len"], s["table"], s["weights"],
                   s["ws"], s["status"], max_q=s["max_q"], add_to=s["before"], causal=c["causal"],
                   window=c["window"])
    return (s["weights"],)


def _own_evict(s):
    from decode_gemv_gb300 import lw
    c = s["case"]
    lw.lw_kv_evict(s["cache"], s["weights"], s["kv_len"], s["table"], s["out_table"], s["out_len"],
                   s["out_weights"], s["kept"], s["status"], keep=c["keep"], first=c["first"],
                   recent=c["recent"])
    slots = _out_slots(s)
    k = torch.empty(slots.shape[0], c["kv_heads"], c["dim"], dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    lw.lw_kv_read(s["cache"], slots, k, v, s["status"])
    return s["kept"], s["out_len"], s["out_weights"], k, v


def _own_blocks(s):
    from decode_gemv_gb300 import lw
    c = s["case"]
    lw.lw_kv_summarise(s["cache"], s["summary"], s["start"], s["kv_len"], s["table"], s["status"])
    lw.lw_kv_attention_blocks(s["cache"], s["summary"], s["q"], s["q_start"], s["kv_len"], s["table"],
                              s["out"], s["ws"], s["status"], blocks=c["blocks"], first=c["first"],
                              recent=c["recent"], chosen=s["chosen"])
    return s["out"], s["chosen"]


def _out_slots(s):
    """Slots of the kept tokens of every sequence, -1 where it has fewer."""
    c, page = s["case"], s["case"]["page"]
    j = torch.arange(c["keep"], device=DEV)
    slots = s["out_table"][:, j // page].long() * page + j % page
    return torch.where(j < s["out_len"][:, None], slots, -1).view(-1)


# ---- plain forms -----------------------------------------------------------

def _plain_quantise(x):
    """Codes [n, h, D], scales and minimums fp16 [n, h, G]."""
    n, h, d = x.shape
    f = x.float().view(n, h, d // GROUP, GROUP)
    bad = ~torch.isfinite(f).all(-1)
    f = f.clamp(-LIMIT, LIMIT)
    low, high = f.amin(-1), f.amax(-1)
    scale, low = ((high - low) * (1 / 15)).half(), low.half()
    s, m = scale.float()[..., None], low.float()[..., None]
    inv = torch.where(s > 0, 1 / s, torch.zeros_like(s))
    codes = torch.round((f - m) * inv).clamp(0, 15)
    codes = torch.where(bad[..., None], torch.zeros_like(codes), codes).to(torch.int32)
    nan = torch.full_like(scale, math.nan)
    return codes.view(n, h, d), torch.where(bad, nan, scale), torch.where(bad, nan, low)


def _units(dim):
    """[16, units of a token]: where token t's 16-bit units lie in its tile: key codes, key
    scales, key minimums, value codes, value scales, value minimums."""
    g, sizes = dim // GROUP, _tile_units(dim)
    at = [sum(sizes[:i]) for i in range(6)]
    gp = g + g % 2
    t = torch.arange(16, device=DEV)[:, None]
    u = torch.arange(dim // 4, device=DEV)[None]
    i = torch.arange(g, device=DEV)[None]
    par = (t // 2 * g + i) * 2 + t % 2
    return torch.cat([at[0] + ((t * 4 + u % 8 // 2) * g + u // 8) * 2 + u % 2,
                      at[1] + par, at[2] + t * gp + i,
                      at[3] + ((t // 2 * 8 + u % 8) * g + u // 8) * 2 + t % 2,
                      at[4] + par, at[5] + par], 1)


def _where(case, slots, head=None):
    """[..., units]: places in the pages, seen as 16-bit units, of slots [n] for every head
    ([n, h, units]) or of slots [..., h, n] of the heads that come with them."""
    dim, heads, page = case["dim"], case["kv_heads"], case["page"]
    size = sum(_tile_units(dim))
    if head is None:
        slots, head = slots[:, None], torch.arange(heads, device=DEV)
    tile = (slots // page * heads + head) * (page // 16) + slots % page // 16
    return tile[..., None] * size + _units(dim)[slots % 16]


def _plain_write(pages, case, k, v, slots):
    parts = []
    shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)
    for x in (k, v):
        codes, scale, low = _plain_quantise(x)
        n, h, d = codes.shape
        packed = (codes.view(n, h, d // 4, 4) << shift).sum(-1).to(torch.int16)
        parts += [packed, scale.view(torch.int16), low.view(torch.int16)]
    # the last page takes what is not stored
    to = torch.where(slots < 0, pages.shape[0] * case["page"] - 1, slots)
    pages.view(-1)[_where(case, to)] = torch.cat(parts, -1)


def _restored(case, units):
    """Keys and values fp32 [..., D] of tokens' units."""
    d, g = case["dim"], case["dim"] // GROUP
    shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)
    out = []
    for x in units.split([d // 4 + 2 * g] * 2, -1):
        codes, scale, low = x.split([d // 4, g, g], -1)
        c = ((codes.to(torch.int32)[..., None] >> shift) & 15).float()
        c = c.reshape(*units.shape[:-1], g, GROUP)
        scale, low = (p.contiguous().view(torch.float16).float()[..., None] for p in (scale, low))
        # (an fp16 scale times 4 bits is exact in fp32: one rounding, by the sum)
        out.append((c * scale + low).reshape(*units.shape[:-1], d))
    return out


def _plain_read(s, slots):
    units = s["pages"].view(-1)[_where(s["case"], slots.clamp(min=0))]
    gone = (slots < 0)[:, None, None]
    return [x.masked_fill(gone, 0.0) for x in _restored(s["case"], units)]


def _rotate(case, x, cos, sin):
    """x fp32 [n, heads, D], cos and sin [n, 1, rot / 2]."""
    rot = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rotary(s):
    case, pos = s["case"], s["pos"]
    cos, sin = s["table"][pos.clamp(min=0)][:, None].chunk(2, -1)
    k = _rotate(case, s["k"].float(), cos, sin)
    q = _rotate(case, s["q"].float(), cos, sin).to(s["q"].dtype)
    _plain_write(s["pages"], case, k, s["v"], s["slots"])
    k, v = _plain_read(s, s["slots"])
    q = torch.where((pos < 0)[:, None, None], s["q_out"], q)
    return q, k.to(s["k"].dtype), v.to(s["v"].dtype)


def _tile_parts(case, tiles):
    """Keys fp32 [..., 16, D] of whole tiles [..., units]."""
    d, g = case["dim"], case["dim"] // GROUP
    lead = tiles.shape[:-1]
    kc, ks, km = tiles.split(_tile_units(d), -1)[:3]
    shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)
    ks = ks.contiguous().view(torch.float16).view(*lead, 8, g, 2).transpose(-1, -2)
    ks = ks.reshape(*lead, 16, g, 1).float()
    km = km.contiguous().view(torch.float16).view(*lead, 16, g + g % 2)[..., :g, None].float()
    kc = (kc.to(torch.int32)[..., None] >> shift) & 15
    kc = kc.reshape(*lead, 16, 4, g, 2, 4).transpose(-3, -4)     # t, g, q, h, i
    return (kc.reshape(*lead, 16, g, GROUP) * ks + km).reshape(*lead, 16, d)


def _plain_keys(s, b=None):
    """Keys of every sequence, fp32 [batch, kv_heads, slots, D], or of one."""
    table = s["table"] if b is None else s["table"][b:b + 1]
    tiles = s["pages"][table.clamp(min=0).long()].transpose(1, 2)       # [b, h, pages, tiles, units]
    k = _tile_parts(s["case"], tiles).flatten(2, 4)
    return k if b is None else k[0]


def _padded(s):
    """Row i of sequence b among the packed tokens [batch, t], and whether there is one."""
    start = s["q_start"].long()
    row = torch.arange(s["max_q"], device=DEV)
    at = start[:-1, None] + row
    return at.clamp(max=s["q"].shape[0] - 1), row < (start[1:] - start[:-1])[:, None]


def _plain_weigh(s):
    case, q, n = s["case"], s["q"], s["kv_len"].long()
    b, hq, h, d, t = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], s["max_q"]
    k = _plain_keys(s)
    width = s["weights"].shape[2]
    k = k[:, :, :width]
    at, there = _padded(s)
    x = q.float()[at].view(b, t, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    lse = s["lse"][at].view(b, t, h, hq // h).permute(0, 2, 3, 1).reshape(b, h, -1, 1)
    col = torch.arange(width, device=DEV)
    pos = (n - there.sum(1))[:, None] + torch.arange(t, device=DEV)
    see = (col < n[:, None, None]) & there[..., None]
    if case["causal"]:
        see = see & (col <= pos[..., None])
    if case["window"]:
        see = see & (col > pos[..., None] - case["window"])
    p = torch.exp((x @ k.transpose(-1, -2)) * (1 / math.sqrt(d)) - lse)
    p = torch.where(see[:, None, None], p.view(b, h, hq // h, t, -1), 0.0)
    w = p.sum((2, 3))
    return (w if s["before"] is None else torch.where(col < n[:, None, None], s["before"] + w, 0.0),)


def _plain_evict(s):
    case, n, w = s["case"], s["kv_len"].long(), s["weights"]
    keep, first, recent, page = case["keep"], case["first"], case["recent"], case["page"]
    col = torch.arange(w.shape[2], device=DEV)
    m = n.clamp(max=keep)
    must = (col < first) | (col >= (n - recent)[:, None])
    w = torch.where(must[:, None], math.inf, w)
    w = torch.where(col < n[:, None, None], w, -1.0)       # (weights are not negative)
    order = w.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    rank = torch.arange(order.shape[-1], device=DEV)
    big = w.shape[2]
    order = torch.where(rank < m[:, None, None], order, big).sort(-1).values
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=big)
    has = order < big
    s["kept"].copy_(torch.where(has, order, -1))
    s["out_len"].copy_(m)
    at = order.clamp(max=big - 1)
    s["out_weights"].copy_(torch.where(has, s["weights"].gather(2, at), 0.0))
    # the kept tokens' units to their new places; the others go where nothing is read
    head = torch.arange(case["kv_heads"], device=DEV)[:, None]
    seq = torch.arange(case["batch"], device=DEV)[:, None, None]
    src = s["table"][seq, at // page].long().clamp(min=0) * page + at % page
    j = torch.arange(keep, device=DEV)
    dst = (s["out_table"][:, j // page].long() * page + j % page)[:, None].expand_as(src)
    units = s["pages"].view(-1)
    units[_where(case, dst, head)] = units[_where(case, src, head)]
    k, v = _plain_read(s, _out_slots(s))
    return s["kept"], s["out_len"], s["out_weights"], k.half(), v.half()


def _plain_summarise(s, start, end, most):
    """Ranges of the keys of the pages that hold tokens start .. end - 1 (at most `most` pages a
    sequence), into s["summary"]."""
    case, page = s["case"], s["case"]["page"]
    first, last = start.long() // page, -(-end.long() // page)
    at = first[:, None] + torch.arange(most, device=DEV)
    seq, i = torch.nonzero((at < last[:, None]) & (start < end)[:, None], as_tuple=True)
    block = at[seq, i]
    page_id = s["table"][seq, block].long()
    k = _tile_parts(case, s["pages"][page_id]).flatten(2, 3)       # [n, h, page, D]
    slot = block[:, None] * page + torch.arange(page, device=DEV)
    there = (slot < end.long()[seq][:, None])[:, None, :, None]
    low = torch.where(there, k, math.inf).amin(2)
    high = torch.where(there, k, -math.inf).amax(2)
    top = torch.maximum(low.abs(), high.abs()).amax(-1, keepdim=True)
    inv = torch.where(top > 2.0 ** -100, 127 / top, torch.zeros_like(top))
    codes = torch.round(torch.stack([high, low], 2) * inv[:, :, None]).to(torch.int8)
    step = (top * torch.tensor(1 / 127, device=DEV)).expand(*top.shape[:2], 4).contiguous()
    step[..., 1:] = 0
    s["summary"][page_id] = torch.cat([codes.flatten(2).view(torch.uint8), step.view(torch.uint8)], -1)


def _choose(s, scores, count):
    """The chosen blocks of each token and head, ascending, -1 where there are fewer."""
    case, col = s["case"], torch.arange(scores.shape[2], device=DEV)
    nb = count[:, None, None]
    must = (col < case["first"]) | (col >= nb - case["recent"])
    scores = torch.where(col < nb, torch.where(must, math.inf, scores), -math.inf)
    take = min(case["blocks"], scores.shape[2])
    order = scores.sort(dim=-1, descending=True, stable=True).indices[..., :take]
    big = scores.shape[2]
    order = torch.where(torch.arange(take, device=DEV) < nb, order, big).sort(-1).values
    order = torch.nn.functional.pad(order, (0, case["blocks"] - take), value=big)
    return torch.where(order < big, order, -1)


def _codes(case, q):
    """Queries as whole numbers up to 127 and their steps, [tokens, kv_heads, group, D or 1]."""
    x = q.float().view(q.shape[0], case["kv_heads"], -1, case["dim"])
    top = x.abs().amax(-1, keepdim=True)
    inv = torch.where(top > 2.0 ** -100, 127 / top, torch.zeros_like(top))
    return torch.round(x * inv), top * torch.tensor(1 / 127, device=DEV)


def _positions(s):
    """Sequence and key position of each packed token."""
    start = s["q_start"].long()
    token = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.bucketize(token, start[1:], right=True)
    return seq, s["kv_len"].long()[seq] - start[seq + 1] + token


def _plain_blocks(s):
    case, d, page = s["case"], s["case"]["dim"], s["case"]["page"]
    new = min(s["table"].shape[1], -(-case["fresh"] // page) + 1)
    _plain_summarise(s, s["start"], s["kv_len"], new)
    seq, pos = _positions(s)
    code, step = _codes(case, s["q"])
    hi = s["summary"][..., :d].view(torch.int8).float()
    lo = s["summary"][..., d:2 * d].view(torch.int8).float()
    unit = s["summary"][..., 2 * d:2 * d + 4].contiguous().view(torch.float32)[..., 0]
    ids = s["table"].clamp(min=0).long()                                  # [b, width]
    hi, lo, unit = (x[ids].transpose(1, 2)[seq] for x in (hi, lo, unit))  # [tokens, h, width, ..]
    # (whole numbers below 2^24: any order of the sums is exact)
    dot = code.clamp(min=0) @ hi.transpose(-1, -2) + code.clamp(max=0) @ lo.transpose(-1, -2)
    scores = (dot * step).amax(2) * unit
    chosen = _choose(s, scores, -(-(pos + 1) // page))
    s["chosen"].copy_(chosen)
    # attention over the chosen pages alone
    n, h = chosen.shape[:2]
    at = chosen.clamp(min=0)
    ids = s["table"][seq[:, None, None], at].long().clamp(min=0)
    tiles = s["pages"][ids, torch.arange(h, device=DEV)[:, None]]        # [tokens, h, blocks, tiles, u]
    k, v = _plain_tiles(case, tiles)
    key = (at[..., None] * page + torch.arange(page, device=DEV))
    see = (chosen[..., None] >= 0) & (key <= pos[:, None, None, None])
    see = see.flatten(2)[:, :, None]
    x = s["q"].float().view(n, h, -1, d)
    score = torch.where(see, (x @ k.transpose(-1, -2)) * (1 / math.sqrt(d)), -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = (p @ torch.where(see.transpose(-1, -2), v, 0.0)) / p.sum(-1, keepdim=True)
    return out.reshape(s["q"].shape).to(s["q"].dtype), s["chosen"]


def _plain_tiles(case, tiles):
    """Keys and values fp32 [tokens, h, keys, D] of whole tiles [tokens, h, blocks, tiles, units]."""
    d, g = case["dim"], case["dim"] // GROUP
    lead = tiles.shape[:-1]
    vc, vs, vm = tiles.split(_tile_units(d), -1)[3:]
    shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)
    vs, vm = (x.contiguous().view(torch.float16).view(*lead, 8, g, 2).transpose(-1, -2)
              .reshape(*lead, 16, g, 1).float() for x in (vs, vm))
    vc = (vc.to(torch.int32)[..., None] >> shift) & 15
    vc = vc.reshape(*lead, 8, 8, g, 2, 4)                                  # t / 2, n, g, t % 2, i
    vc = vc.movedim(-2, -4).transpose(-3, -2)                              # t / 2, t % 2, g, n, i
    v = vc.reshape(*lead, 16, g, GROUP) * vs + vm
    return _tile_parts(case, tiles).flatten(2, 4), v.reshape(*lead, 16, d).flatten(2, 4)


# ----------------------------------------------------------------------------
# the definition, in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "weigh": _exact_weigh, "evict": _exact_evict,
            "blocks": _exact_blocks}[case["op"]](s)


def _exact_rotary(s):
    case, pos, rot = s["case"], s["pos"], s["case"]["rot"]
    row = s["table"].double()[pos.clamp(min=0)]
    turn = torch.complex(row[:, :rot // 2], row[:, rot // 2:])[:, None]

    def pairs(x):
        z = x[..., :rot]
        return z.unflatten(-1, (-1, 2)) if case["interleaved"] else \
            z.unflatten(-1, (2, -1)).transpose(-1, -2)

    def placed(x, z):
        y = x.double().clone()
        y[..., :rot] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return y

    z = torch.view_as_complex(pairs(s["q"].double()).contiguous())
    q = placed(s["q"], torch.view_as_real(z * turn))
    q[pos < 0] = 0
    # which code a value gets is defined in fp32, step by step: each step in 64 bits, then rounded
    a, b = pairs(s["k"].double()).unbind(-1)
    c, d = turn.real, turn.imag
    z = torch.stack([_fp32(_fp32(a * c) - _fp32(b * d)), _fp32(_fp32(b * c) + _fp32(a * d))], -1)
    out = [q]
    for x in (placed(s["k"], z), s["v"].double()):
        f = x.view(x.shape[0], x.shape[1], -1, GROUP)
        low, high = f.aminmax(dim=-1, keepdim=True)
        scale = _fp32(_fp32(high - low) * _fp32(torch.tensor(1 / 15, dtype=torch.float64, device=DEV)))
        scale, low = scale.half().double(), low.half().double()
        inv = torch.where(scale > 0, _fp32(1 / scale), 0.0)
        code = _fp32(_fp32(f - low) * inv).round().clamp(0, 15)
        y = (scale * code + low).view(x.shape)
        y[s["slots"] < 0] = 0
        out.append(y)
    return tuple(out)


def _fp32(x):
    return x.float().double()


def _exact_token(s, page_id, head, pos):
    """Keys and values fp64 [n, D] of n slots of pages, element by element from the bytes."""
    case = s["case"]
    d, page = case["dim"], case["page"]
    g = d // GROUP
    sizes = [2 * u for u in _tile_units(d)]
    base = [sum(sizes[:i]) for i in range(6)]
    byts = s["pages"].view(torch.uint8).view(-1)
    half = s["pages"].view(torch.float16).view(-1)
    pos = pos[:, None]
    j = torch.arange(d, device=DEV)[None]
    tile = (page_id.long()[:, None] * case["kv_heads"] + head) * (page // 16)
    tile = (tile + pos % page // 16) * sum(sizes)
    t, grp, r = pos % 16, j // 32, j % 32
    kbyte = base[0] + 4 * ((t * 4 + r // 8) * g + grp) + r % 8 // 2
    vbyte = base[3] + 4 * ((t // 2 * 8 + r // 4) * g + grp) + 2 * (t % 2) + r % 4 // 2
    par = 4 * (t // 2 * g + grp) + 2 * (t % 2)
    got = []
    for code, scale, low in ((kbyte, base[1] + par, base[2] + 2 * (t * (g + g % 2) + grp)),
                             (vbyte, base[4] + par, base[5] + par)):
        c = (byts[tile + code].long() >> (4 * (j % 2))) & 15
        got.append(half[(tile + scale) // 2].double() * c + half[(tile + low) // 2].double())
    return got


def _exact_weigh(s):
    case, q = s["case"], s["q"]
    group, page = case["q_heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
    start = s["q_start"].tolist()
    for b, n in enumerate(s["kv_len"].tolist()):
        t = start[b + 1] - start[b]
        pos = torch.arange(n, device=DEV)
        see = _visible(case, t, n) if n and t else None
        for h in range(case["kv_heads"]):
            if n and t:
                k, _ = _exact_token(s, s["table"][b, pos // page], h, pos)
                for i in range(h * group, (h + 1) * group):
                    x = q[start[b]:start[b + 1], i].double() @ k.T / math.sqrt(case["dim"])
                    x = (x - s["lse"][start[b]:start[b + 1], i, None].double()).exp()
                    out[b, h, :n] += x.masked_fill(~see, 0.0).sum(0)
            if s["before"] is not None:
                out[b, h, :n] += s["before"][b, h, :n].double()
    return (out,)


def _exact_evict(s):
    case, page = s["case"], s["case"]["page"]
    keep, heads = case["keep"], case["kv_heads"]
    kept = torch.full(s["kept"].shape, -1, dtype=torch.int64, device=DEV)
    weights = torch.zeros(s["out_weights"].shape, dtype=torch.float64, device=DEV)
    k = torch.zeros(case["batch"], keep, heads, case["dim"], dtype=torch.float64, device=DEV)
    v = torch.zeros_like(k)
    for b, n in enumerate(s["kv_len"].tolist()):
        m = min(n, keep)
        for h in range(heads if m else 0):
            w = s["weights"][b, h, :n].double()
            rank = torch.where(w == w, w, math.inf)
            rank[max(0, n - case["recent"]):] = math.inf
            rank[:case["first"]] = math.inf
            limit = rank.sort(descending=True).values[m - 1]
            sure = rank > limit
            tied = torch.nonzero(rank == limit)[:, 0][:m - int(sure.sum())]
            sure[tied] = True
            at = torch.nonzero(sure)[:, 0]
            kept[b, h, :m], weights[b, h, :m] = at, w[at]
            k[b, :m, h], v[b, :m, h] = _exact_token(s, s["table"][b, at // page], h, at)
    lens = s["kv_len"].long().clamp(max=keep)
    return kept, lens, weights, k.flatten(0, 1), v.flatten(0, 1)


def _exact_blocks(s):
    case, page, d = s["case"], s["case"]["page"], s["case"]["dim"]
    group, heads = case["q_heads"] // case["kv_heads"], case["kv_heads"]
    seq, pos = _positions(s)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    chosen = torch.full(s["chosen"].shape, -1, dtype=torch.int64, device=DEV)
    code, step = _codes(case, s["q"])     # (the codes are defined in fp32)
    old = None
    for i in range(s["q"].shape[0]):
        b, p = int(seq[i]), int(pos[i])
        nb, n = p // page + 1, int(s["kv_len"][b])
        if old != b:
            ranges, old = [_exact_ranges(s, b, h, n) for h in range(heads)], b
        for h in range(heads):
            codes, unit = ranges[h]
            c = code[i, h].double()[:, None]
            dot = torch.maximum(c * codes[0], c * codes[1])[:, :nb].sum(-1)
            score = ((dot.float() * step[i, h]).amax(0) * unit[:nb]).double()
            score[max(0, nb - case["recent"]):] = math.inf
            score[:case["first"]] = math.inf
            take = min(nb, case["blocks"])
            limit = score.sort(descending=True).values[take - 1]
            sure = score > limit
            sure[torch.nonzero(score == limit)[:, 0][:take - int(sure.sum())]] = True
            at = torch.nonzero(sure)[:, 0]
            chosen[i, h, :take] = at
            key = (at[:, None] * page + torch.arange(page, device=DEV)).view(-1)
            key = key[key <= p]
            k, v = _exact_token(s, s["table"][b, key // page], h, key)
            x = s["q"][i, h * group:(h + 1) * group].double() @ k.T / math.sqrt(d)
            out[i, h * group:(h + 1) * group] = x.softmax(-1) @ v
    return out, chosen


def _exact_ranges(s, b, h, n):
    """Codes [2][blocks, D] and steps [blocks] of one head's pages (defined in fp32)."""
    page, d = s["case"]["page"], s["case"]["dim"]
    nb = -(-n // page)
    at = torch.arange(n, device=DEV)
    k = _exact_token(s, s["table"][b, at // page], h, at)[0].float()
    k = torch.cat([k, k[-1:].expand(nb * page - n, d)]).view(nb, page, d)
    ends = torch.stack([k.amax(1), k.amin(1)])
    top = ends.abs().amax((0, 2))[:, None]
    inv = torch.where(top > 2.0 ** -100, 127 / top, torch.zeros_like(top))
    return torch.round(ends * inv).double(), (top * torch.tensor(1 / 127, device=DEV))[:, 0]
