"""Plain implementations, in 64 bits on the cached values, of what the calls around the 4-bit
key/value cache compute; shared by their GPU tests."""
import math

import torch

from decode_gemv_gb300 import lw

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pool(gen, n_pages, heads, dim, page):
    """A cache in memory that holds any bits."""
    size = n_pages * lw.lw_kv_page_bytes(heads, dim, page)
    return lw.KvCache(torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV, generator=gen), heads, dim, page)


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def keys_values(gen, n, heads, dim):
    k = torch.randn(n, heads, dim, device=DEV, generator=gen)
    v = torch.randn(n, heads, dim, device=DEV, generator=gen)
    k[..., 3] = 3 * k[..., 3] + 4
    return k, v


def filled(gen, lens, heads, dim, page, spare=0):
    """A pool, its page table (-1 past a sequence's pages) with lens[b] written tokens a sequence, and the ids of
    spare + 1 further pages."""
    used = [-(-n // page) for n in lens]
    cache = pool(gen, sum(used) + spare + 1, heads, dim, page)
    order = torch.randperm(cache.n_pages, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(max(used), 1)), -1, dtype=torch.int32, device=DEV)
    at, st = 0, status()
    for b, n in enumerate(lens):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        if n:
            k, v = keys_values(gen, n, heads, dim)
            lw.lw_kv_write(cache, k, v, slots_of(table[b], range(n), page), st)
    torch.cuda.synchronize()
    assert int(st) == 0
    return cache, table, order[at:]


def slots_of(row, tokens, page):
    t = torch.tensor(list(tokens), dtype=torch.int64, device=DEV)
    return row.long()[t // page] * page + t % page


def read(cache, slots):
    """Cached keys and values, fp32 [n, heads, dim]."""
    k = torch.empty(slots.shape[0], cache.kv_heads, cache.head_dim, device=DEV)
    v, st = torch.empty_like(k), status()
    lw.lw_kv_read(cache, slots, k, v, st)
    return k, v


def read_all(cache):
    """Every slot of the pool, as bits."""
    k, v = read(cache, torch.arange(cache.n_pages * cache.page_tokens, device=DEV))
    return torch.stack([k, v]).view(torch.int32)


def spans(T, n, causal=True, window=0):
    """Which of n keys each of T tokens sees, bool [T, n]."""
    pos = torch.arange(n - T, n, device=DEV)[:, None]
    key = torch.arange(n, device=DEV)[None]
    see = torch.ones(T, n, dtype=torch.bool, device=DEV)
    if causal:
        see &= key <= pos
    if window:
        see &= key > pos - window
    return see


def scores(q, k, see, scale):
    """fp64 scores [T, q_heads, n] of queries [T, q_heads, D] and keys [n, heads, D], -inf where unseen."""
    group = q.shape[1] // k.shape[1]
    s = torch.einsum("thd,jhd->thj", q.double(), k.double().repeat_interleave(group, 1)) * scale
    return s.masked_fill(~see[:, None], -math.inf)


def relative(x, y):
    x, y = x.double(), y.double()
    return float((x - y).norm() / y.norm().clamp(min=1e-300))
