"""The key/value cache operators: what they compute, at the sizes they are used at.

A token generator keeps the keys and values of past tokens next to its coded
weights.  Two operators hold them in 4 bits:

* the cache's write and read-back (lw_kv_write, lw_kv_read): each token's keys
  and values are quantised as they are stored -- 4-bit codes with an fp16
  scale and minimum per 32 values -- and read back as scale * code + minimum;
* attention over that cache (lw_kv_attention): the queries of a batch of
  sequences of any lengths, one token each or many, against the 4-bit pages.

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
        # one decode step of one sequence: the new token's keys and values, as
        # the fp32 outputs of the coded k and v products
        dict(name="cache 1 token fp32", op="cache", tokens=1, kv_heads=8, dim=128, page=64,
             type="fp32", skip=0),
        # one decode step of a padded batch: scattered slots, some of them
        # padding that is not stored
        dict(name="cache 61 tokens fp32", op="cache", tokens=61, kv_heads=32, dim=96, page=16,
             type="fp32", skip=5),
        # a prompt of odd length
        dict(name="cache 5003 tokens bf16", op="cache", tokens=5003, kv_heads=8, dim=128, page=64,
             type="bf16", skip=0),
        # a long prompt, or a cache moved between machines
        dict(name="cache 131072 tokens bf16", op="cache", tokens=131072, kv_heads=8, dim=128,
             page=256, type="bf16", skip=0),
        # the first token after a short prompt: latency alone
        dict(name="decode 1x37 fp32", op="attention", batch=1, q_heads=32, kv_heads=8, dim=128,
             page=64, type="fp32", q_min=1, q_max=1, len_min=37, len_max=37, window=0,
             causal=True, lse=False, past=False, shape=1),
        # one sequence in the middle of an answer
        dict(name="decode 1x4097 fp32", op="attention", batch=1, q_heads=32, kv_heads=8, dim=128,
             page=64, type="fp32", q_min=1, q_max=1, len_min=4097, len_max=4097, window=0,
             causal=True, lse=False, past=False, shape=2),
        # a served batch of ragged lengths, empty slots among them
        dict(name="decode 64 ragged bf16", op="attention", batch=64, q_heads=32, kv_heads=8,
             dim=128, page=64, type="bf16", q_min=1, q_max=1, len_min=0, len_max=4096, window=0,
             causal=True, lse=False, past=False, shape=3),
        # few sequences with very long contexts
        dict(name="decode 8 long bf16", op="attention", batch=8, q_heads=32, kv_heads=8, dim=128,
             page=256, type="bf16", q_min=1, q_max=1, len_min=20000, len_max=131072, window=0,
             causal=True, lse=False, past=False, shape=4),
        # checking five drafted tokens of each of 16 sequences, a head of keys
        # for every head of queries
        dict(name="draft 16x5 fp32", op="attention", batch=16, q_heads=32, kv_heads=32, dim=96,
             page=16, type="fp32", q_min=5, q_max=5, len_min=200, len_max=2500, window=0,
             causal=True, lse=False, past=False, shape=5),
        # a chunk of a long prompt on what is in the cache already
        dict(name="chunk 2048 on 14336 bf16", op="attention", batch=1, q_heads=32, kv_heads=8,
             dim=128, page=64, type="bf16", q_min=2048, q_max=2048, len_min=14336, len_max=14336,
             window=0, causal=True, lse=False, past=True, shape=6),
        # several whole prompts, a sliding window over the newest 1024 keys
        dict(name="prompts window fp16", op="attention", batch=5, q_heads=16, kv_heads=2, dim=64,
             page=32, type="fp16", q_min=1, q_max=4095, len_min=0, len_max=0, window=1024,
             causal=True, lse=False, past=True, shape=7),
        # short chunks in fp32, with the row sums for a later merge
        dict(name="chunk 2x90 fp32", op="attention", batch=2, q_heads=32, kv_heads=8, dim=128,
             page=64, type="fp32", q_min=70, q_max=90, len_min=2000, len_max=2600, window=0,
             causal=True, lse=True, past=True, shape=8),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["cache", "decode", "decode", "chunk"])
    dim = rng.choice([64, 96, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if kind == "cache":
        typ = rng.choice(["fp32", "bf16", "bf16", "fp16"])
        top = 131072 * 8 * 128 // (kv_heads * dim * (2 if typ == "fp32" else 1))
        return dict(op="cache", tokens=_log(rng, 1, min(131072, top)), kv_heads=kv_heads, dim=dim,
                    page=page, type=typ, skip=rng.choice([0, 0, 7]))
    group = rng.choice([1, 1, 2, 4, 4, 8]) if kv_heads < 32 else 1
    case = dict(op="attention", batch=1, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                page=page, type=rng.choice(["fp32", "bf16", "bf16", "fp16"]), q_min=1, q_max=1,
                len_min=0, len_max=0, window=rng.choice([0, 0, 0, 129, 4096]), causal=True,
                lse=rng.random() < 0.25, past=kind == "chunk",
                shape=rng.randrange(1 << 20))
    if kind == "decode":
        case["q_max"] = rng.choice([1, 1, 1, 2, 4, 7])
        case["batch"] = _log(rng, 1, 200)
        # the padded cache, and the scores, stay within the listed ones
        top = min(131072, (1 << 30) // (case["batch"] * kv_heads * dim * case["q_max"]))
        case["len_max"] = max(1, _log(rng, 1, max(2, top)))
        case["len_min"] = rng.choice([0, 1, case["len_max"] // 8, case["len_max"]])
        case["causal"] = rng.random() < 0.8
    else:
        case["q_max"] = _log(rng, 9, 4096)
        case["q_min"] = rng.choice([0, case["q_max"] // 2, case["q_max"]])
        case["batch"] = _log(rng, 1, 6)
        # products and scores of the padded batch within the listed ones
        rows = case["batch"] * case["q_heads"] * case["q_max"]
        top = min(32768, (1 << 29) // rows)
        past = max(0, top - case["q_max"])
        case["len_max"] = _log(rng, 1, past) if past > 1 else 0
        case["len_min"] = rng.choice([0, case["len_max"] // 2, case["len_max"]])
    return case


def _lengths(case):
    """Query tokens and cached keys (the new tokens' own among them) of each sequence."""
    rng = random.Random(case["shape"])
    q, kv = [], []
    for _ in range(case["batch"]):
        t = rng.randint(case["q_min"], case["q_max"])
        n = rng.randint(case["len_min"], case["len_max"])
        q.append(t)
        # a chunk comes on top of what is cached; a decode step's length counts its own tokens
        kv.append(n + t if case["past"] else n)
    q[0], kv[0] = max(q[0], 1), max(kv[0], 1)
    return q, kv


def _tile_units(dim):
    """16-bit units of the six parts of a tile of 16 tokens."""
    g = dim // GROUP
    return [4 * dim, 16 * g, 16 * (g + g % 2), 4 * dim, 16 * g, 16 * g]


def work(case):
    """Inputs once, outputs once; of the cache the codes, scales and minimums that the call
    writes and reads, or those of the keys that some query of the call may see."""
    d, h = case["dim"], case["kv_heads"]
    size = 4 if case["type"] == "fp32" else 2
    token = 2 * h * (d // 2 + 4 * (d // GROUP))   # cached bytes of one token
    if case["op"] == "cache":
        n = case["tokens"]
        kept = n - (n // case["skip"] if case["skip"] else 0)
        return {"bytes": kept * (2 * h * d * size + 2 * token) + n * (2 * h * d * size + 8),
                "flops": 8.0 * 2 * kept * h * d}
    byts, pairs = 0, 0
    for t, n in zip(*_lengths(case)):
        first = max(0, n - t - case["window"] + 1) if case["window"] else 0
        byts += 2 * t * case["q_heads"] * d * size + (token * (n - first) if t and n else 0)
        byts += (4 * t * case["q_heads"] if case["lse"] else 0) + 4 * -(-n // case["page"])
        # keys that the tokens may see, summed
        for lo, hi in _spans(case, t, n):
            pairs += hi - lo
    return {"bytes": byts, "flops": 4.0 * case["q_heads"] * d * pairs}


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


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    typ = TYPES[case["type"]]
    if case["op"] == "cache":
        n, page = case["tokens"], case["page"]
        k, v = _keys_values(gen, n, case["kv_heads"], case["dim"])
        pages = -(-n // page) + 1
        # runs of 16 slots in any order, as pages are handed out
        runs = torch.randperm((pages - 1) * (page // 16), device=DEV, generator=gen)
        slots = (runs[:, None] * 16 + torch.arange(16, device=DEV)).reshape(-1)[:n].contiguous()
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1
        state = dict(case=case, k=k.to(typ), v=v.to(typ), slots=slots,
                     pages=_stale(gen, _page_shape(case, pages)))
    else:
        state = _attention_state(case, gen, typ)
    if own:   # the handle, workspace and status word that a user's program keeps
        from decode_gemv_gb300 import lw
        state["cache"] = lw.KvCache(state["pages"].view(torch.uint8), case["kv_heads"],
                                    case["dim"], case["page"])
        state["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if case["op"] == "attention":
            need = lw.lw_kv_workspace_bytes(state["cache"], case["q_heads"], state["q"].shape[0],
                                            case["batch"])
            state["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return state


def _attention_state(case, gen, typ):
    q_len, kv_len = _lengths(case)
    page, batch = case["page"], case["batch"]
    used = [-(-n // page) for n in kv_len]
    width = max(max(used), 1)
    pages = sum(used) + 3
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
    q = torch.randn(sum(q_len), case["q_heads"], case["dim"], device=DEV, generator=gen)
    start = torch.tensor([0] + q_len, device=DEV).cumsum(0).to(torch.int32)
    lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    q = (1.5 * q).to(typ)
    return dict(case=case, pages=store, q=q, q_start=start, kv_len=lens, table=table,
                max_q=max(q_len), out=torch.empty_like(q),
                lse=torch.empty(q.shape[:2], device=DEV) if case["lse"] else None)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    if own:
        return _own_cache(state) if state["case"]["op"] == "cache" else _own_attention(state)
    return _plain_cache(state) if state["case"]["op"] == "cache" else _plain_attention(state)


def _own_cache(s):
    from decode_gemv_gb300 import lw
    lw.lw_kv_write(s["cache"], s["k"], s["v"], s["slots"], s["status"])
    k, v = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    lw.lw_kv_read(s["cache"], s["slots"], k, v, s["status"])
    return k, v


def _own_attention(s):
    from decode_gemv_gb300 import lw
    c = s["case"]
    lw.lw_kv_attention(s["cache"], s["q"], s["q_start"], s["kv_len"], s["table"], s["out"],
                       s["ws"], s["status"], max_q=s["max_q"], causal=c["causal"],
                       window=c["window"], lse=s["lse"])
    return (s["out"], s["lse"]) if c["lse"] else (s["out"],)


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


def _where(case, slots):
    """[n, h, units]: places in the pages, seen as 16-bit units."""
    dim, heads, page = case["dim"], case["kv_heads"], case["page"]
    size = sum(_tile_units(dim))
    head = torch.arange(heads, device=DEV)
    tile = (slots // page)[:, None] * heads + head
    tile = tile * (page // 16) + (slots % page // 16)[:, None]
    return tile[..., None] * size + _units(dim)[slots % 16][:, None, :]


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


def _plain_cache(s):
    case = s["case"]
    _plain_write(s["pages"], case, s["k"], s["v"], s["slots"])
    slots = s["slots"]
    units = s["pages"].view(-1)[_where(case, slots.clamp(min=0))]
    n, h, d, g = slots.shape[0], case["kv_heads"], case["dim"], case["dim"] // GROUP
    shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)
    back = []
    for x in units.split([d // 4 + 2 * g] * 2, -1):
        codes, scale, low = x.split([d // 4, g, g], -1)
        c = ((codes.to(torch.int32)[..., None] >> shift) & 15).float().view(n, h, g, GROUP)
        scale, low = (p.contiguous().view(torch.float16).float()[..., None] for p in (scale, low))
        f = (c * scale + low).view(n, h, d)
        back.append(torch.where((slots < 0)[:, None, None], torch.zeros_like(f), f))
    return back[0].to(s["k"].dtype), back[1].to(s["v"].dtype)


def _plain_gather(s):
    """Keys and values of every sequence, fp32 [batch, kv_heads, slots, D]."""
    case = s["case"]
    d, h, g = case["dim"], case["kv_heads"], case["dim"] // GROUP
    tiles = s["pages"][s["table"].clamp(min=0).long()]       # [b, pages, h, tiles, units]
    b = tiles.shape[0]
    tiles = tiles.transpose(1, 2).reshape(b, h, -1, tiles.shape[-1])
    kc, ks, km, vc, vs, vm = tiles.split(_tile_units(d), -1)
    shift = torch.arange(0, 16, 4, device=DEV, dtype=torch.int32)

    def paired(x):      # [t / 2][g][t % 2] -> [t, g]
        x = x.contiguous().view(torch.float16).view(b, h, -1, 8, g, 2).transpose(-1, -2)
        return x.reshape(b, h, -1, g, 1).float()

    km = km.contiguous().view(torch.float16).view(b, h, -1, g + g % 2)[..., :g, None].float()
    kc = (kc.to(torch.int32)[..., None] >> shift) & 15
    kc = kc.reshape(b, h, -1, 4, g, 2, 4).transpose(-3, -4)     # t, g, q, h, i
    k = kc.reshape(b, h, -1, g, GROUP) * paired(ks) + km
    vc = (vc.to(torch.int32)[..., None] >> shift) & 15
    vc = vc.reshape(b, h, -1, 8, g, 2, 4).permute(0, 1, 2, 5, 4, 3, 6)   # pairs, t % 2, g, n, i
    v = vc.reshape(b, h, -1, g, GROUP) * paired(vs) + paired(vm)
    return k.reshape(b, h, -1, d), v.reshape(b, h, -1, d)


def _plain_attention(s):
    case, q, n = s["case"], s["q"], s["kv_len"].long()
    b, hq, h, d, t = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], s["max_q"]
    start = s["q_start"].long()
    k, v = _plain_gather(s)
    row = torch.arange(t, device=DEV)
    count = start[1:] - start[:-1]
    at = (start[:-1, None] + row).clamp(max=q.shape[0] - 1)
    x = q.float()[at].view(b, t, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    col = torch.arange(k.shape[2], device=DEV)
    pos = (n - count)[:, None] + row
    see = (col < n[:, None, None]).expand(b, t, -1)
    if case["causal"]:
        see = see & (col <= pos[..., None])
    if case["window"]:
        see = see & (col > pos[..., None] - case["window"])
    score = (x @ k.transpose(-1, -2)).view(b, h, hq // h, t, -1) * (1 / math.sqrt(d))
    score = torch.where(see[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where((col < n[:, None])[:, None, :, None], v, 0.0)
    out = (p.view(b, h, -1, p.shape[-1]) @ v).view(b, h, hq // h, t, d)
    out = torch.where(total > 0, out / total, torch.where(total == 0, 0.0, total))
    lse = (top + torch.log(total))[..., 0]
    # back to the packed tokens
    token = torch.arange(q.shape[0], device=DEV)
    seq = torch.bucketize(token, start[1:], right=True)
    i = token - start[seq]
    out = out.permute(0, 3, 1, 2, 4)[seq, i].reshape(q.shape).to(q.dtype)
    lse = lse.permute(0, 3, 1, 2)[seq, i].reshape(q.shape[:2])
    return (out, lse) if case["lse"] else (out,)


# ----------------------------------------------------------------------------
# the definition, in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_cache(s) if case["op"] == "cache" else _exact_attention(s)


def _exact_cache(s):
    out = []
    for x in (s["k"], s["v"]):
        f = x.double().view(x.shape[0], x.shape[1], -1, GROUP)
        low, high = f.aminmax(dim=-1, keepdim=True)
        scale, low = ((high - low) / 15).half().double(), low.half().double()
        c = ((f - low) / scale).nan_to_num(0.0).round().clamp(0, 15)
        y = (scale * c + low).view(x.shape)
        y[s["slots"] < 0] = 0
        out.append(y)
    return tuple(out)


def _exact_rows(s, b, head):
    """Keys and values of one sequence's head: fp64 [n, D], element by element from the bytes."""
    case = s["case"]
    n, d, page = int(s["kv_len"][b]), case["dim"], case["page"]
    g = d // GROUP
    sizes = [2 * u for u in _tile_units(d)]
    base = [sum(sizes[:i]) for i in range(6)]
    byts = s["pages"].view(torch.uint8).view(-1)
    half = s["pages"].view(torch.float16).view(-1)
    pos = torch.arange(n, device=DEV)[:, None]
    j = torch.arange(d, device=DEV)[None]
    tile = (s["table"][b, pos // page].long() * case["kv_heads"] + head) * (page // 16)
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


def _exact_attention(s):
    case, q = s["case"], s["q"]
    group = case["q_heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    start = s["q_start"].tolist()
    for b, n in enumerate(s["kv_len"].tolist()):
        t = start[b + 1] - start[b]
        if not t or not n:
            continue
        pos = torch.arange(n - t, n, device=DEV)[:, None]
        key = torch.arange(n, device=DEV)[None]
        hidden = torch.zeros(t, n, dtype=torch.bool, device=DEV)
        if case["causal"]:
            hidden |= key > pos
        if case["window"]:
            hidden |= key <= pos - case["window"]
        for h in range(case["kv_heads"]):
            k, v = _exact_rows(s, b, h)
            for i in range(h * group, (h + 1) * group):
                x = q[start[b]:start[b + 1], i].double() @ k.T / math.sqrt(case["dim"])
                x.masked_fill_(hidden, -math.inf)
                z = x.logsumexp(-1, keepdim=True)
                out[start[b]:start[b + 1], i] = (x - z).exp().nan_to_num(0.0) @ v
                lse[start[b]:start[b + 1], i] = z[:, 0]
    return (out, lse) if case["lse"] else (out,)
