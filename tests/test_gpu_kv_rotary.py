"""Rotary positions on the GPU: the table against its formulas in 64 bits; the rotating cache write against
lw_kv_write of keys that the same fp32 steps rotated (every byte of the pages), and its queries against those steps.

Both are exact: the definition fixes each fp32 operation, and rounds queries once.  The table is one rounding to
fp32 of a fp64 value whose angle is off by at most 2^-52 p f: 2^-24 relative to the value and 1e-9 absolute at these
positions."""
import math

import numpy as np
import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from kv_plain import DEV, TYPES, generator, keys_values, pool, read_all, status


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def frequencies(rot, kind, base, factor, old, low, high):
    """By the formulas, with a loop a pair."""
    if kind == lw.LW_ROTARY_NTK and rot > 2:
        base *= factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if kind == lw.LW_ROTARY_LINEAR:
            f /= factor
        elif kind == lw.LW_ROTARY_BANDS:
            k = min(1.0, max(0.0, (old * f / (2 * math.pi) - low) / (high - low)))
            f *= k + (1 - k) / factor
        elif kind == lw.LW_ROTARY_YARN:
            def pair(turns):
                return rot * math.log(old / (2 * math.pi * turns)) / (2 * math.log(base))
            a, b = max(0, math.floor(pair(high))), min(rot - 1, math.ceil(pair(low)))
            k = 1 - min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            f *= k + (1 - k) / factor
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("rot", [2, 34, 128])
@pytest.mark.parametrize("kind,kw", [
    (lw.LW_ROTARY_PLAIN, dict(base=10000.0)), (lw.LW_ROTARY_LINEAR, dict(base=500000.0, factor=4.0)),
    (lw.LW_ROTARY_NTK, dict(base=10000.0, factor=8.0)),
    (lw.LW_ROTARY_BANDS, dict(base=500000.0, factor=8.0, old_length=8192.0)),
    (lw.LW_ROTARY_BANDS, dict(base=10000.0, factor=2.0, old_length=300.0, low=0.5, high=40.0, gain=0.75)),
    (lw.LW_ROTARY_YARN, dict(base=10000.0, factor=16.0, old_length=4096.0)),
    (lw.LW_ROTARY_YARN, dict(base=10000.0, factor=16.0, old_length=4096.0, low=2.0, high=20.0, gain=1.0))])
@pytest.mark.parametrize("first,n", [(0, 1), (0, 130), (123456, 77)])
def test_table(rot, kind, kw, first, n):
    table = torch.full((n, rot), 9.0, device=DEV)
    lw.lw_rotary_table(table, first=first, scaling=kind, **kw)
    yarn = kind == lw.LW_ROTARY_YARN
    f = frequencies(rot, kind, kw["base"], kw.get("factor", 1.0), kw.get("old_length", 1.0), kw.get("low", 0) or 1.0,
                    kw.get("high", 0) or (32.0 if yarn else 4.0))
    gain = kw.get("gain", 0) or (0.1 * math.log(kw["factor"]) + 1 if yarn else 1.0)
    a = (first + np.arange(n))[:, None] * f
    want = np.concatenate([np.cos(a), np.sin(a)], 1) * gain
    assert (np.abs(table.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 1e-9).all()


def rotated(x, row, rot, near):
    """x fp32 [n, heads, D], row [n, rot]: the definition's fp32 steps."""
    c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
    y = x.clone()
    ia = torch.arange(0, rot, 2, device=DEV) if near else torch.arange(rot // 2, device=DEV)
    ib = ia + (1 if near else rot // 2)
    a, b = x[..., ia], x[..., ib]
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    y[..., ia] = ac - bs
    y[..., ib] = bc + as_
    return y


CASES = [   # n, q heads, kv heads, dim, page, rot, near, skipped tokens
    (1, 32, 8, 128, 64, 128, False, ()), (1, 1, 1, 64, 16, 64, True, ()),
    (17, 6, 3, 96, 48, 96, False, (3, 16)), (33, 4, 4, 96, 16, 48, True, (0,)),
    (70, 5, 1, 128, 128, 32, False, ()), (70, 8, 2, 64, 32, 6, True, (1, 2, 69)),
    (40, 3, 3, 128, 16, 126, False, ()), (19, 2, 1, 64, 16, 2, False, ()),
    (300, 32, 8, 128, 64, 64, True, ()), (31, 9, 9, 96, 16, 90, True, (30,)),
]


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("layout", ["apart", "in place", "packed", "odd"])
def test_write(typ, case, layout):
    n, hq, h, dim, page, rot, near, skipped = case
    gen, st = generator(n * 7 + rot), status()
    k, v = (x.to(TYPES[typ]) for x in keys_values(gen, n, h, dim))
    q = torch.randn(n, hq, dim, device=DEV, generator=gen).to(TYPES[typ])
    if layout == "packed":     # one product's output: queries, keys, values of a token side by side
        buf = torch.cat([q, k, v], 1)
        q, k, v = buf[:, :hq], buf[:, hq:hq + h], buf[:, hq + h:]
    elif layout == "odd":      # rows that start on no 16-byte boundary
        def odd(x):
            y = torch.zeros(x.shape[0], x.shape[1], dim + 3, dtype=x.dtype, device=DEV)[..., 1:dim + 1]
            return y.copy_(x)
        q, k, v = odd(q), odd(k), odd(v)
    positions = torch.randint(0, 5000, (n,), device=DEV, generator=gen)
    table = torch.empty(5000, rot, device=DEV)
    lw.lw_rotary_table(table, base=1000.0)
    a = pool(gen, -(-n // page) + 1, h, dim, page)
    b = lw.KvCache(a.pages.clone(), h, dim, page)
    slots = torch.randperm(a.n_pages * page, device=DEV, generator=gen)[:n].contiguous()
    q0, k0, v0 = (x.float().contiguous() for x in (q, k, v))
    out = torch.full((n, hq, dim), 7.0, dtype=TYPES[typ], device=DEV) if layout in ("apart", "odd") else q
    want_q = rotated(q0, table[positions], rot, near).to(TYPES[typ])
    before = out.clone()
    to = slots.clone()
    for i, t in enumerate(skipped):
        if i % 2:              # not stored, rotated all the same
            slots[t] = to[t] = -1
        else:                  # skipped
            positions[t], to[t] = -1, -1
            want_q[t] = before[t]
    lw.lw_kv_write_rotary(a, k, v, slots, positions, table, st, q=q, q_out=out, interleaved=near)
    lw.lw_kv_write(b, rotated(k0, table[positions.clamp(min=0)], rot, near), v0, to, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert torch.equal(a.pages, b.pages)
    assert torch.equal(out, want_q)
    c = lw.KvCache(b.pages.clone(), h, dim, page)     # without queries: the same cache
    if layout != "packed" and layout != "in place":
        lw.lw_kv_write_rotary(c, k, v, slots, positions, table, st, interleaved=near)
        assert torch.equal(c.pages, b.pages)


def test_positions_past_the_table_and_slots_past_the_pages():
    gen, st = generator(3), status()
    n, h, dim, page, rot = 20, 2, 64, 16, 64
    k, v = keys_values(gen, n, h, dim)
    q = torch.randn(n, 4, dim, device=DEV, generator=gen)
    table = torch.empty(100, rot, device=DEV)
    lw.lw_rotary_table(table)
    a = pool(gen, 3, h, dim, page)
    before = read_all(a)
    out = torch.full_like(q, 5.0)
    slots, pos = torch.arange(n, device=DEV), torch.arange(n, device=DEV)
    pos[4] = 100
    lw.lw_kv_write_rotary(a, k, v, slots, pos, table, st, q=q, q_out=out)
    assert int(st) == lw.LW_DEV_BAD_POSITION
    assert torch.equal(read_all(a)[:, 4], before[:, 4]) and bool((out[4] == 5).all())
    assert torch.equal(out[5], rotated(q, table[pos.clamp(max=99)], rot, False)[5])
    pos[4], slots[6], st = 4, 48, status()
    lw.lw_kv_write_rotary(a, k, v, slots, pos, table, st, q=q, q_out=out)
    assert int(st) == lw.LW_DEV_BAD_SLOT
    assert torch.equal(out, rotated(q, table[pos], rot, False))    # (its queries are rotated)
    lw.lw_kv_write_rotary(a, k, v, slots, pos, table[:0], st, q=q, q_out=out)     # no positions at all
    assert torch.equal(out, rotated(q, table[pos], rot, False))
    z = torch.empty(0, dtype=torch.int64, device=DEV)
    lw.lw_kv_write_rotary(a, k[:0], v[:0], z, z, table, st, q=q[:0], q_out=out[:0])


def test_values_that_are_not_finite():
    gen, st = generator(4), status()
    k, v = keys_values(gen, 16, 1, 64)
    k[3, 0, 5], k[4, 0, 40], k[5, 0, 2] = math.nan, math.inf, 1e30
    table = torch.empty(16, 64, device=DEV)
    lw.lw_rotary_table(table)
    pos = torch.arange(16, device=DEV)
    a = pool(gen, 1, 1, 64, 16)
    b = lw.KvCache(a.pages.clone(), 1, 64, 16)
    lw.lw_kv_write_rotary(a, k, v, pos, pos, table, st)
    lw.lw_kv_write(b, rotated(k, table, 64, False), v, pos, st)
    assert int(st) == 0 and torch.equal(a.pages, b.pages)
    assert bool(torch.isnan(read_all(a).view(torch.float32)[0, 3]).any())


def test_replayed_on_another_stream():
    gen, st = generator(5), status()
    n, h, dim = 50, 2, 128
    k, v = keys_values(gen, n, h, dim)
    q = torch.randn(n, 8, dim, device=DEV, generator=gen)
    first = q.clone()
    table = torch.empty(400, dim, device=DEV)
    lw.lw_rotary_table(table)
    pos, slots = torch.arange(n, device=DEV), torch.arange(n, device=DEV)
    a = pool(gen, 4, h, dim, 16)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = lw.StepGraph(side)
    with g.capture():
        lw.lw_kv_write_rotary(a, k, v, slots, pos, table, st, q=q, q_out=out)
    for shift in (0, 100, 350):
        pos.copy_(torch.arange(n, device=DEV) + shift)
        q.copy_(first * (1 + shift))
        torch.cuda.synchronize()
        g.launch()
        torch.cuda.synchronize()
        assert torch.equal(out, rotated(q, table[pos], dim, False))
    assert int(st) == 0
