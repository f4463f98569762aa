"""The 4-bit key/value cache on the GPU: lw_kv_write / lw_kv_read against the
definition, lw_kv_attention against a plain implementation in 64 bits on the
cached values, over types, head counts, lengths, masks, page sizes and
strides; what a corrupt page table or length does.

Tolerances, from the arithmetic (u = unit roundoff of the output type, 2^-24
fp32, 2^-11 fp16, 2^-8 bf16):
* the cache: the kernel's operations are the definition's, so written codes,
  scales and minimums are equal; a value read back is one rounded fp32 fma,
  then one rounding to the type: equal to the same steps in numpy.
* attention, normwise over a head row set (2-norm of the difference over the
  2-norm of the result): scores of magnitude S = max |s| are computed to
  2^-22 S at least (fp32 sums of 22-bit products), so p to 2^-21 S; values
  enter as scale * code + min whose parts are up to 4 times |v| in these
  inputs; with S <= 40 here the result is within 4 * 40 * 2^-21 = 7.6e-5 in
  fp32 and fp16 (16-bit operands carried in two parts), plus u.  bf16 calls
  may round the operands of the products to 11 bits: scores to
  2^-11 * S_rms (rounding errors of 64..128 products add as their root:
  S_rms <= 6 here), values and p to 2^-11: 1e-2 in all, plus u.
"""
import math

import numpy as np
import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
TOL = {"fp32": 7.6e-5, "fp16": 7.6e-5 + 2.0 ** -11, "bf16": 1e-2 + 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---- the definition, in numpy ----------------------------------------------

def quantise(x):
    """x fp32 [n, h, D] -> codes, scale, min (fp16) of groups of 32."""
    n, h, d = x.shape
    f = x.reshape(n, h, d // 32, 32).astype(np.float32)
    bad = ~np.isfinite(f).all(-1)
    f = np.clip(np.nan_to_num(f, nan=0.0, posinf=np.inf, neginf=-np.inf), -61440, 61440).astype(np.float32)
    lo, hi = f.min(-1), f.max(-1)
    scale = ((hi - lo) * np.float32(1.0 / 15.0)).astype(np.float16)
    low = lo.astype(np.float16)
    s, m = scale.astype(np.float32)[..., None], low.astype(np.float32)[..., None]
    with np.errstate(divide="ignore"):
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0))
    c = np.clip(np.rint((f - m) * inv), 0, 15).astype(np.int64)
    c[bad] = 0
    scale[bad] = np.nan
    low[bad] = np.nan
    return c, scale, low


def dequantise(c, scale, low):
    n, h, g, _ = c.shape
    y = c * scale.astype(np.float64)[..., None] + low.astype(np.float64)[..., None]
    return y.reshape(n, h, g * 32)


def tile_fields(tile, dim):
    """Codes [16, D], scales and minimums [16, G] of keys and values, entry by entry from the
    documented places of a tile's bytes."""
    g = dim // 32
    gp = g + g % 2
    u8, f16 = tile, tile.view(np.float16)
    at = np.cumsum([0, 8 * dim, 32 * g, 32 * gp, 8 * dim, 32 * g])
    out = {n: np.zeros((16, dim), np.int64) for n in ("kc", "vc")}
    out.update({n: np.zeros((16, g), np.float16) for n in ("ks", "km", "vs", "vm")})
    for t in range(16):
        for d in range(dim):
            grp, r = d // 32, d % 32
            b = at[0] + 4 * ((t * 4 + r // 8) * g + grp) + (r % 8) // 2
            out["kc"][t, d] = (u8[b] >> (4 * (r % 2))) & 15
            b = at[3] + 4 * ((t // 2 * 8 + r // 4) * g + grp) + 2 * (t % 2) + (r % 4) // 2
            out["vc"][t, d] = (u8[b] >> (4 * (r % 2))) & 15
        for grp in range(g):
            pair = (t // 2 * g + grp) * 2 + t % 2
            out["ks"][t, grp] = f16[at[1] // 2 + pair]
            out["km"][t, grp] = f16[at[2] // 2 + t * gp + grp]
            out["vs"][t, grp] = f16[at[4] // 2 + pair]
            out["vm"][t, grp] = f16[at[5] // 2 + pair]
    return out


def make_kv(rng, n, heads, dim):
    k = rng.standard_normal((n, heads, dim)).astype(np.float32)
    v = rng.standard_normal((n, heads, dim)).astype(np.float32)
    k[..., 3] = 3 * k[..., 3] + 4
    return k, v


# ---- write and read --------------------------------------------------------

@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("n,heads,dim,page", [(1, 1, 64, 16), (17, 3, 96, 48), (40, 8, 128, 32),
                                              (333, 2, 128, 256)])
def test_write_is_the_definition_and_read_returns_it(typ, n, heads, dim, page):
    rng = np.random.default_rng(7 * n + dim)
    k, v = (torch.from_numpy(a).to(DEV).to(TYPES[typ]) for a in make_kv(rng, n, heads, dim))
    pages = -(-n // page) + 1
    cache = lw.KvCache(torch.randint(0, 256, (pages * lw.lw_kv_page_bytes(heads, dim, page),),
                                     dtype=torch.uint8, device=DEV), heads, dim, page)
    slots = torch.from_numpy(rng.permutation(pages * page)[:n].astype(np.int64)).to(DEV)
    if n > 16:
        slots[5] = -1
    before = cache.pages.cpu().numpy().copy()
    st = status()
    lw.lw_kv_write(cache, k, v, slots, st)
    ko, vo = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    lw.lw_kv_read(cache, slots, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    raw = cache.pages.cpu().numpy()
    tb = lw.lw_kv_tile_bytes(dim)
    tiles = raw.reshape(pages, heads, page // 16, tb)
    sl = slots.cpu().numpy()
    want = {"k": quantise(k.float().cpu().numpy()), "v": quantise(v.float().cpu().numpy())}
    # every cached field, at its documented place
    seen = {}
    for i, s in enumerate(sl):
        if s < 0:
            continue
        for h in range(heads):
            key = (s // page, h, s % page // 16)
            if key not in seen:
                seen[key] = tile_fields(tiles[key], dim)
            f, t = seen[key], s % 16
            for n_, w in (("k", want["k"]), ("v", want["v"])):
                assert np.array_equal(f[n_ + "c"][t], w[0][i, h].reshape(-1))
                assert np.array_equal(f[n_ + "s"][t], w[1][i, h])
                assert np.array_equal(f[n_ + "m"][t], w[2][i, h])
    # nothing else changed: write the same tokens' bytes back to `before` through the fields'
    # places would repeat the layout, so count instead -- bytes that differ lie in written tiles
    diff = (before != raw).reshape(pages, heads, page // 16, tb).any(-1)
    for p, h, t in zip(*np.nonzero(diff)):
        assert (p, h, t) in seen
    for got, w in ((ko, want["k"]), (vo, want["v"])):
        y = dequantise(*w).astype(np.float32)   # scale * code is exact, one rounding to fp32
        y[sl < 0] = 0
        assert torch.equal(got.cpu(), torch.from_numpy(y).to(TYPES[typ]))


def test_a_token_owns_its_bytes():
    """Tokens of one tile written by different calls do not disturb each other."""
    rng = np.random.default_rng(3)
    k, v = (torch.from_numpy(a).to(DEV) for a in make_kv(rng, 32, 2, 96))
    a = lw.KvCache(torch.zeros(2 * lw.lw_kv_page_bytes(2, 96, 16), dtype=torch.uint8, device=DEV), 2, 96, 16)
    b = lw.KvCache(torch.zeros_like(a.pages), 2, 96, 16)
    st = status()
    slots = torch.arange(32, device=DEV)
    lw.lw_kv_write(a, k, v, slots, st)
    for i in rng.permutation(32):
        i = int(i)
        lw.lw_kv_write(b, k[i:i + 1], v[i:i + 1], slots[i:i + 1], st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert torch.equal(a.pages, b.pages)


def test_values_that_are_hard_to_hold():
    n, d = 8, 64
    x = np.zeros((n, 1, d), np.float32)
    x[1] = 3.25                                  # one value: scale 0
    x[2, 0, :] = np.linspace(-1e30, 1e30, d)     # beyond fp16: held as +-61440
    x[3, 0, 5] = np.nan
    x[4, 0, 40] = np.inf
    x[5, 0, :] = 1e-9 * np.arange(d)             # scale underflows to 0
    x[6, 0, :] = -0.0
    x[7, 0, :32] = np.linspace(-61440, 61440, 32)
    k = torch.from_numpy(x).to(DEV)
    cache = lw.KvCache.empty(1, 1, d, 16)
    st, slots = status(), torch.arange(n, device=DEV)
    lw.lw_kv_write(cache, k, k.clone(), slots, st)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    lw.lw_kv_read(cache, slots, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    want = dequantise(*quantise(x)).astype(np.float32)
    for o in (ko, vo):
        np.testing.assert_array_equal(o.cpu().numpy(), want)
    got = ko.cpu().numpy()
    assert np.isnan(got[3, 0, :32]).all() and np.isfinite(got[3, 0, 32:]).all()
    assert np.isnan(got[4, 0, 32:]).all() and np.isfinite(got[4, 0, :32]).all()
    assert np.isfinite(got[[0, 1, 2, 5, 6, 7]]).all()
    assert got[2].max() <= 65504 and got[2].min() == -61440


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
def test_strided_and_unaligned_rows(typ):
    """Rows inside a wider tensor (a fused product's output), heads outermost, odd offsets."""
    rng = np.random.default_rng(11)
    n, heads, dim = 21, 4, 96
    k, v = (torch.from_numpy(a).to(DEV).to(TYPES[typ]) for a in make_kv(rng, n, heads, dim))
    ref = lw.KvCache(torch.zeros(2 * lw.lw_kv_page_bytes(heads, dim, 16), dtype=torch.uint8, device=DEV),
                     heads, dim, 16)
    st, slots = status(), torch.arange(n, device=DEV)
    lw.lw_kv_write(ref, k, v, slots, st)
    fused = torch.zeros(n, 2 * heads * dim + 1, device=DEV, dtype=TYPES[typ])
    fk = fused[:, 1:1 + heads * dim].view(n, heads, dim)
    fv = fused[:, 1 + heads * dim:].view(n, heads, dim)
    fk.copy_(k)
    fv.copy_(v)
    outer = [torch.empty(heads, n, dim, device=DEV, dtype=TYPES[typ]).transpose(0, 1) for _ in range(2)]
    outer[0].copy_(k)
    outer[1].copy_(v)
    for a, b in ((fk, fv), tuple(outer)):
        c = lw.KvCache(torch.zeros_like(ref.pages), heads, dim, 16)
        lw.lw_kv_write(c, a, b, slots, st)
        torch.cuda.synchronize()
        assert torch.equal(c.pages, ref.pages)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    lw.lw_kv_read(ref, slots, ko, vo, st)
    for a, b in ((fk, fv), tuple(outer)):
        a.zero_()
        b.zero_()
        lw.lw_kv_read(ref, slots, a, b, st)
        torch.cuda.synchronize()
        assert torch.equal(a, ko) and torch.equal(b, vo)
    assert int(st) == 0 and float(fused[:, 0].abs().max()) == 0


def test_slots_past_the_pages_are_reported():
    cache = lw.KvCache(torch.zeros(lw.lw_kv_page_bytes(1, 64, 16), dtype=torch.uint8, device=DEV), 1, 64, 16)
    k = torch.ones(3, 1, 64, device=DEV)
    st = status()
    slots = torch.tensor([16, -5, 1 << 60], device=DEV)
    lw.lw_kv_write(cache, k, k, slots, st)
    torch.cuda.synchronize()
    assert int(st) == lw.LW_DEV_BAD_SLOT and int(cache.pages.sum()) == 0
    st.zero_()
    o = torch.full_like(k, 7.0)
    lw.lw_kv_read(cache, slots, o, o.clone(), st)
    torch.cuda.synchronize()
    assert int(st) == lw.LW_DEV_BAD_SLOT and float(o.abs().max()) == 0


def test_no_tokens():
    cache = lw.KvCache.empty(1, 1, 64, 16)
    z = torch.empty(0, 1, 64, device=DEV)
    st, slots = status(), torch.empty(0, dtype=torch.int64, device=DEV)
    lw.lw_kv_write(cache, z, z, slots, st)
    lw.lw_kv_read(cache, slots, z, z, st)
    torch.cuda.synchronize()
    assert int(st) == 0


# ---- attention -------------------------------------------------------------

class Setup:
    """A cache of sequences of the given lengths in shuffled pages over stale memory, queries,
    and the cached values in fp64."""

    def __init__(self, seed, q_len, kv_len, q_heads, kv_heads, dim, page, typ, q_gain=1.5,
                 v_gain=1.0):
        rng = np.random.default_rng(seed)
        self.args = (q_heads, kv_heads, dim, page)
        self.q_len, self.kv_len, self.typ = q_len, kv_len, typ
        used = [-(-n // page) for n in kv_len]
        width = max(max(used), 1)
        total = sum(used) + 2
        self.cache = lw.KvCache(torch.randint(0, 256, (total * lw.lw_kv_page_bytes(kv_heads, dim, page),),
                                              dtype=torch.uint8, device=DEV), kv_heads, dim, page)
        order = rng.permutation(total).astype(np.int32)
        table = np.full((len(kv_len), width), -1, np.int32)
        at, self.k, self.v, self.st = 0, [], [], status()
        for b, n in enumerate(kv_len):
            table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            k, v = make_kv(rng, n, kv_heads, dim)
            v = (v * v_gain).astype(np.float32)
            pos = np.arange(n)
            slots = table[b, pos // page].astype(np.int64) * page + pos % page if n else pos.astype(np.int64)
            lw.lw_kv_write(self.cache, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV),
                           torch.from_numpy(slots).to(DEV), self.st)
            self.k.append(dequantise(*quantise(k)))
            self.v.append(dequantise(*quantise(v)))
        self.table = torch.from_numpy(table).to(DEV)
        q = (q_gain * rng.standard_normal((sum(q_len), q_heads, dim))).astype(np.float32)
        self.q = torch.from_numpy(q).to(DEV).to(TYPES[typ])
        self.start = torch.from_numpy(np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)).to(DEV)
        self.lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)

    def run(self, causal=True, window=0, scale=None, lse=True, max_q=None, stream=None, ws=None,
            q=None, out=None):
        q_heads = self.args[0]
        q = self.q if q is None else q
        out = torch.full_like(self.q, 5.0) if out is None else out
        l = torch.full((self.q.shape[0], q_heads), 5.0, device=DEV) if lse else None
        if ws is None:
            ws = torch.zeros(lw.lw_kv_workspace_bytes(self.cache, q_heads, self.q.shape[0],
                                                      len(self.kv_len)), dtype=torch.uint8, device=DEV)
        lw.lw_kv_attention(self.cache, q, self.start, self.lens, self.table, out, ws, self.st,
                           max_q=max(self.q_len) if max_q is None else max_q, scale=scale,
                           causal=causal, window=window, lse=l, stream=stream)
        return out, l

    def want(self, causal=True, window=0, scale=None):
        q_heads, kv_heads, dim, _ = self.args
        scale = dim ** -0.5 if scale is None else scale
        q = self.q.double().cpu().numpy()
        out = np.zeros(q.shape)
        lse = np.full(q.shape[:2], -np.inf)
        at = 0
        for b, (t, n) in enumerate(zip(self.q_len, self.kv_len)):
            pos = np.arange(n - t, n)[:, None]
            j = np.arange(n)[None]
            see = np.ones((t, n), bool)
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            for h in range(q_heads):
                kh = h // (q_heads // kv_heads)
                if t and n:
                    s = scale * (q[at:at + t, h] @ self.k[b][:, kh].T)
                    s = np.where(see, s, -np.inf)
                    m = s.max(-1, keepdims=True)
                    m = np.where(np.isfinite(m), m, 0)
                    p = np.exp(s - m)
                    l = p.sum(-1, keepdims=True)
                    with np.errstate(divide="ignore", invalid="ignore"):
                        out[at:at + t, h] = np.where(l > 0, p @ self.v[b][:, kh] / l, 0)
                        lse[at:at + t, h] = (m + np.log(l))[:, 0]
            at += t
        return out, lse

    def check(self, **kw):
        got, lse = self.run(**kw)
        torch.cuda.synchronize()
        assert int(self.st) == 0
        want, wl = self.want(**{k: v for k, v in kw.items() if k in ("causal", "window", "scale")})
        close(got, want, self.typ)
        if lse is not None:
            lse = lse.double().cpu().numpy()
            assert np.array_equal(np.isfinite(lse), np.isfinite(wl))
            f = np.isfinite(wl)
            # scores to the operand rounding, |s| <= 40: absolute
            if f.any():
                assert np.abs(lse[f] - wl[f]).max() <= 40 * (2.0 ** -10 if self.typ == "bf16" else 2.0 ** -20)
        return got


def close(got, want, typ):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    empty = ~want.any(-1)
    assert not g[empty].any()
    norm = np.linalg.norm(want)
    err = np.linalg.norm(g - want)
    assert err <= TOL[typ] * norm + 1e-300, f"{err / norm:.3e}"
    if norm:   # and no single row is lost in the sum: 8 times the bound, row by row
        rows = np.linalg.norm(want, axis=-1)
        rerr = np.linalg.norm(g - want, axis=-1)
        assert (rerr <= 8 * TOL[typ] * np.maximum(rows, 0.05 * rows.max())).all()


HEADS = [(1, 1, 64), (4, 4, 96), (8, 2, 128), (16, 2, 64), (12, 4, 96), (32, 1, 128), (7, 1, 128)]


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
def test_single_tokens(typ, q_heads, kv_heads, dim):
    """One new token a sequence; lengths of zero and one, around tiles and pages."""
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 257, 1000]
    Setup(1, [1] * len(lens), lens, q_heads, kv_heads, dim, 64, typ).check()


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("typ", ["fp32", "bf16"])
def test_page_sizes(typ, page):
    Setup(2, [1, 2, 1, 3], [5, 300, 48, 777], 8, 2, 128, page, typ).check()


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
@pytest.mark.parametrize("batch,n", [(1, 9000), (2, 4099)])
def test_long_axis_split(typ, batch, n):
    """Few rows, a long axis: the work of a row is split and joined."""
    Setup(3, [1] * batch, [n - 7 * i for i in range(batch)], 8, 2, 128, 64, typ).check()


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50), (False, 130)])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(4, 4, 96), (8, 2, 128), (8, 1, 64)])
def test_few_tokens(typ, causal, window, q_heads, kv_heads, dim):
    """Several tokens a sequence, none for some; more tokens than keys (rows that see nothing)."""
    Setup(4, [5, 0, 3, 7, 1, 6], [100, 40, 3, 4, 260, 0], q_heads, kv_heads, dim, 32, typ).check(
        causal=causal, window=window)


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100), (False, 333)])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(2, 2, 96), (8, 2, 128), (8, 1, 64), (6, 2, 128)])
def test_many_tokens(typ, causal, window, q_heads, kv_heads, dim):
    """Chunks of prompts: odd lengths, past keys, no past, more tokens than keys."""
    Setup(5, [129, 1, 65, 0, 200, 40], [700, 300, 65, 10, 90, 41], q_heads, kv_heads, dim, 64, typ).check(
        causal=causal, window=window)


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
def test_long_chunk(typ):
    Setup(6, [300], [5000], 4, 1, 128, 64, typ).check()


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("q_len,kv_len", [([1, 1], [70, 300]), ([40, 90], [100, 400])])
def test_result_does_not_depend_on_the_hint_or_the_call(typ, q_len, kv_len):
    """Equal bits when a call is repeated, also on a workspace that was used before."""
    s = Setup(7, q_len, kv_len, 8, 2, 128, 16, typ)
    ws = torch.zeros(lw.lw_kv_workspace_bytes(s.cache, 8, sum(q_len), len(kv_len)), dtype=torch.uint8,
                     device=DEV)
    a, la = s.run(ws=ws)
    b, lb = s.run(ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)
    for hint in (1, 4096):   # max_q chooses the kernel, not the answer
        s.check(max_q=hint)


def test_scale_and_large_scores():
    s = Setup(8, [1, 9], [500, 200], 4, 2, 64, 16, "fp32", q_gain=6.0)
    s.check(scale=0.5 * 64 ** -0.5)
    s.check(scale=-0.1)
    got, _ = s.run(scale=0.0)
    torch.cuda.synchronize()
    close(got, s.want(scale=0.0)[0], "fp32")


@pytest.mark.parametrize("gain", [1e-4, 3000.0])
def test_small_and_large_magnitudes(gain):
    """Queries and values far from 1: no part of the arithmetic leaves its range."""
    s = Setup(9, [1, 20], [200, 90], 4, 2, 64, 16, "fp32", q_gain=1.5 / gain, v_gain=gain)
    s.check(scale=gain * 64 ** -0.5)


def test_strided_queries_and_outputs():
    s = Setup(10, [3, 1, 30], [50, 40, 90], 4, 2, 96, 16, "bf16")
    want, _ = s.run()
    wide = torch.zeros(s.q.shape[0], 3, 4, 97, device=DEV, dtype=s.q.dtype)
    q = wide[:, 1, :, 1:]
    q.copy_(s.q)
    out = torch.zeros(4, s.q.shape[0], 96, device=DEV, dtype=s.q.dtype).transpose(0, 1)
    s.run(q=q, out=out)
    torch.cuda.synchronize()
    assert int(s.st) == 0 and torch.equal(out, want)


def test_on_another_stream():
    s = Setup(11, [2, 40], [100, 60], 8, 2, 128, 16, "bf16")
    want, _ = s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got, _ = s.run()
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("q_len", [[1, 1, 1], [40, 33, 64]])
def test_captured_in_a_step_graph(q_len):
    s = Setup(12, q_len, [130, 64, 70], 8, 2, 128, 16, "bf16")
    want, _ = s.run(lse=False)
    torch.cuda.synchronize()
    out = torch.zeros_like(want)
    ws = torch.zeros(lw.lw_kv_workspace_bytes(s.cache, 8, sum(q_len), 3), dtype=torch.uint8, device=DEV)
    g = lw.StepGraph(torch.cuda.Stream())
    with g.capture():
        s.run(lse=False, out=out, ws=ws)
    for _ in range(3):
        g.launch()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and int(s.st) == 0


@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("q_len", [[1, 1], [40, 70]])
def test_nan_stays_in_its_place(where, q_len):
    """A NaN in a visible key, value or query reaches exactly the rows that see it; masked
    places reach none (stale memory holds any bits in every test here)."""
    s = Setup(13, q_len, [50, 90], 4, 2, 64, 16, "fp32")
    clean, _ = s.run()
    at = int(s.start[1])
    if where == "q":
        s.q[at, 1, 3] = float("nan")
    else:
        x = torch.zeros(1, 2, 64, device=DEV)
        x[0, 0, 3] = float("nan")
        page = int(s.table[1, 60 // 16])
        ok = torch.zeros(1, 2, 64, device=DEV)
        lw.lw_kv_write(s.cache, x if where == "k" else ok, x if where == "v" else ok,
                       torch.tensor([page * 16 + 60 % 16], device=DEV), s.st)
    got, _ = s.run()
    torch.cuda.synchronize()
    nan = torch.isnan(got).any(-1).cpu().numpy()
    t = q_len[1]
    pos = 90 - t + np.arange(t)
    want = np.zeros(nan.shape, bool)
    if where == "q":
        want[at, 1] = True
    else:
        want[at:, :2] = (pos >= 60)[:, None]
    assert np.array_equal(nan, want)
    assert torch.equal(got[:at], clean[:at])


def test_bad_pages_and_lengths_are_reported():
    s = Setup(14, [1, 1], [100, 50], 4, 2, 64, 16, "fp32")
    want, _ = s.run()
    torch.cuda.synchronize()
    table = s.table.clone()
    for bad in (-1, s.cache.n_pages, 2 ** 31 - 1):
        s.st.zero_()
        s.table[0, 2] = bad
        got, _ = s.run()
        torch.cuda.synchronize()
        assert int(s.st) == lw.LW_DEV_BAD_PAGE
        assert torch.equal(got[1], want[1]) and bool(torch.isfinite(got).all())
        # the page's keys are left out
        keep = np.r_[0:32, 48:100]
        kept = Setup(14, [1, 1], [100, 50], 4, 2, 64, 16, "fp32")
        kept.k[0], kept.v[0], kept.kv_len = kept.k[0][keep], kept.v[0][keep], [len(keep), 50]
        close(got, kept.want()[0], "fp32")
    s.table.copy_(table)
    for lens in ([-3, 50], [s.table.shape[1] * 16 + 1, 50]):
        s.st.zero_()
        s.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        got, _ = s.run()
        torch.cuda.synchronize()
        assert int(s.st) == lw.LW_DEV_BAD_SEQ
        assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("start", [[0, 3, 2], [-1, 1, 2], [0, 1, 3]])
def test_bad_query_ranges_are_reported(start):
    s = Setup(15, [1, 1], [100, 50], 4, 2, 64, 16, "fp32")
    s.start.copy_(torch.tensor(start, dtype=torch.int32))
    out = torch.full_like(s.q, 5.0)
    s.run(out=out)
    torch.cuda.synchronize()
    assert int(s.st) == lw.LW_DEV_BAD_SEQ and bool(torch.isfinite(out).all())


def test_no_queries():
    s = Setup(16, [0, 0], [10, 0], 4, 2, 64, 16, "fp32")
    s.run()
    torch.cuda.synchronize()
    assert int(s.st) == 0


def test_many_sequences():
    lens = [(37 * i) % 90 for i in range(700)]
    Setup(17, [1] * 700, lens, 2, 1, 64, 16, "bf16").check()


@pytest.mark.parametrize("typ", ["fp16", "bf16"])
def test_short_and_long_chunks_together(typ):
    """Many items of one key tile between long ones: parts of the kernel that have no work in the
    short ones keep their place."""
    kv_len = [20, 33, 900, 17, 40, 18, 64, 1300, 50, 19] * 6
    Setup(19, [17] * 60, kv_len, 8, 4, 64, 16, typ).check()


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
def test_long_window(typ):
    """Prompts under a sliding window: rows that see nothing of an item's first keys."""
    Setup(20, [700, 900], [700, 1100], 8, 1, 64, 32, typ).check(window=200)


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
def test_many_row_tiles(typ):
    """Prompts of over a hundred row tiles a head between short ones: the search for a CTA's range
    shares them among lanes."""
    Setup(21, [2100, 3, 0, 900], [2100, 50, 9, 1000], 8, 1, 64, 32, typ).check(window=100)


@pytest.mark.parametrize("typ", ["fp16", "bf16"])
def test_long_prompts_among_many_sequences(typ):
    """More sequences than a CTA has threads, two of them of many row tiles."""
    q_len, kv_len = [i % 3 for i in range(700)], [(37 * i) % 90 for i in range(700)]
    for b, t in ((3, 400), (690, 300)):
        q_len[b] = kv_len[b] = t
    Setup(22, q_len, kv_len, 8, 2, 64, 16, typ).check()


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("tokens", [2, 4, 5, 6, 7, 12, 13])
def test_rows_around_the_variants(typ, tokens):
    """8 query heads on 2: 8, 16, 20, 24, 28, 48 and 52 rows of a sequence."""
    Setup(23, [tokens, 1, tokens], [700, 40, tokens], 8, 2, 96, 16, typ).check()


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
@pytest.mark.parametrize("hint", [1, 3, 1000])
def test_any_hint_is_right(typ, hint):
    """max_q below and above the longest sequence's tokens."""
    Setup(24, [1, 77, 30], [300, 500, 30], 8, 2, 128, 32, typ).check(max_q=hint)


def test_offsets_past_32_bits():
    """A cache of over 4 GiB: pages at its far end are written, read and attended."""
    heads, dim, page = 8, 128, 256
    pb = lw.lw_kv_page_bytes(heads, dim, page)
    n_pages = (5 << 30) // pb
    cache = lw.KvCache.empty(n_pages, heads, dim, page)
    cache.pages.fill_(255)
    rng = np.random.default_rng(5)
    k, v = make_kv(rng, 300, heads, dim)
    table = np.array([[n_pages - 1, 0]], np.int32)
    pos = np.arange(300)
    slots = torch.from_numpy(table[0, pos // page].astype(np.int64) * page + pos % page).to(DEV)
    st = status()
    kd, vd = torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV)
    lw.lw_kv_write(cache, kd, vd, slots, st)
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    lw.lw_kv_read(cache, slots, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    np.testing.assert_array_equal(ko.cpu().numpy(), dequantise(*quantise(k)).astype(np.float32))
    for t in (1, 150):
        s = Setup(18, [t], [300], 8, heads, dim, page, "fp32")
        s.cache, s.table = cache, torch.from_numpy(table).to(DEV)
        s.k, s.v = [dequantise(*quantise(k))], [dequantise(*quantise(v))]
        s.check()
