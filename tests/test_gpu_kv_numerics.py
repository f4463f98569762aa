"""Attention over the 4-bit cache on rows that are hard to add up, against a
plain implementation in 64 bits on the cached values: value scales that rise
after a NaN, rows that one key dominates, value groups of very different
scales, and where a NaN goes, element by element.

Tolerances, normwise (u = half a unit of the output type), S = the largest
|score| of a test's inputs (natural units):
* fp32 and fp16 calls: scores and probabilities in 22 bits, 4 S 2^-21 as the
  rest of the tests have it (test_gpu_kv.py), plus u;
* bf16 calls: p and p sc (few rows), p and v (many rows) each rounded to 11
  bits, 2 2^-12; a key of many rows is rounded to 11 bits as well, which where
  its elements err alike moves a score by S 2^-12; plus u = 2^-9.
"""
import numpy as np
import pytest

from decode_gemv_gb300 import lw
from test_gpu_kv import DEV, TYPES, Setup, dequantise, quantise, status

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -9}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def bound(typ, top, many):
    if typ == "bf16":
        return U[typ] + 2.0 ** -11 + (top * 2.0 ** -12 if many else 4 * top * 2.0 ** -21)
    return U[typ] + 4 * top * 2.0 ** -21


class Given(Setup):
    """Sequences of the given keys and values [n, kv_heads, dim] and queries [tokens, q_heads, dim]; the
    very array of the sequence before: the same pages."""

    def __init__(self, k, v, q, page, typ, seed=0):
        kv_heads, dim = k[0].shape[1:]
        rng = np.random.default_rng(seed)
        self.args = (q[0].shape[1], kv_heads, dim, page)
        self.q_len, self.kv_len, self.typ = [len(x) for x in q], [len(x) for x in k], typ
        same = [b > 0 and k[b] is k[b - 1] for b in range(len(k))]
        used = [0 if same[b] else -(-n // page) for b, n in enumerate(self.kv_len)]
        self.cache = lw.KvCache(torch.randint(0, 256, (sum(used) * lw.lw_kv_page_bytes(kv_heads, dim, page),),
                                              dtype=torch.uint8, device=DEV), kv_heads, dim, page)
        order, at = rng.permutation(sum(used)).astype(np.int32), 0
        table = np.full((len(k), max(used)), -1, np.int32)
        self.k, self.v, self.st = [], [], status()
        for b, n in enumerate(self.kv_len):
            if same[b]:
                table[b] = table[b - 1]
                self.k.append(self.k[-1])
                self.v.append(self.v[-1])
                continue
            table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            pos = np.arange(n)
            slots = table[b, pos // page].astype(np.int64) * page + pos % page
            put = [torch.from_numpy(np.ascontiguousarray(x[b], dtype=np.float32)).to(DEV) for x in (k, v)]
            lw.lw_kv_write(self.cache, *put, torch.from_numpy(slots).to(DEV), self.st)
            self.k.append(dequantise(*quantise(np.float32(k[b]))))
            self.v.append(dequantise(*quantise(np.float32(v[b]))))
        self.table = torch.from_numpy(table).to(DEV)
        self.q = torch.from_numpy(np.concatenate(q).astype(np.float32)).to(DEV).to(TYPES[typ])
        self.start = torch.from_numpy(np.concatenate([[0], np.cumsum(self.q_len)]).astype(np.int32)).to(DEV)
        self.lens = torch.tensor(self.kv_len, dtype=torch.int32, device=DEV)

    def expect(self, causal=True, window=0):
        """out (NaN where a NaN of a seen key's value or of its score goes), lse, the largest |score|."""
        q_heads, kv_heads, dim, _ = self.args
        q = self.q.double()
        out, lse, at, top = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV), 0, 0.0
        for b, (t, n) in enumerate(zip(self.q_len, self.kv_len)):
            if not b or self.k[b] is not self.k[b - 1]:
                keys, values = torch.from_numpy(self.k[b]).to(DEV), torch.from_numpy(self.v[b]).to(DEV)
            pos, j = torch.arange(n - t, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
            see = torch.ones(t, n, dtype=torch.bool, device=DEV)
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            for h in range(q_heads):
                k, v = keys[:, h // (q_heads // kv_heads)], values[:, h // (q_heads // kv_heads)]
                s = dim ** -0.5 * (q[at:at + t, h] @ k.nan_to_num(0.0).T)
                top = max(top, float(s[see].abs().max()))
                s = torch.where(see, s, -np.inf)
                e = s.logsumexp(-1)
                o = (s - e[:, None]).exp() @ v.nan_to_num(0.0)
                o[(see.double() @ v.isnan().double()) > 0] = np.nan
                lost = see[:, k.isnan().any(-1)].any(-1)
                o[lost], e[lost] = np.nan, np.nan
                out[at:at + t, h], lse[at:at + t, h] = o, e
            at += t
        return out.cpu().numpy(), lse.cpu().numpy(), top

    def check(self, causal=True, window=0, many=False, group=None, magnitude=None, **kw):
        got, lse = self.run(causal=causal, window=window, **kw)
        torch.cuda.synchronize()
        assert int(self.st) == 0
        want, wl, top = self.expect(causal, window)
        top = top if magnitude is None else magnitude
        g, e = got.double().cpu().numpy(), lse.double().cpu().numpy()
        wrong = int((np.isnan(g) != np.isnan(want)).sum()), int((np.isnan(e) != np.isnan(wl)).sum())
        assert wrong == (0, 0), f"NaN, or none, in {wrong} places of out and lse"
        wrong = int(np.isinf(g).sum())
        assert wrong == 0, f"{wrong} infinities"
        tol = bound(self.typ, top, many)
        d = np.nan_to_num(g) - np.nan_to_num(want)
        for i in range(0, want.shape[-1], group or want.shape[-1]):
            part = np.s_[..., i:i + (group or want.shape[-1])]
            norm = np.linalg.norm(np.nan_to_num(want[part]))
            err = np.linalg.norm(d[part]) / norm if norm else 0.0
            assert err <= tol, f"from element {i}: {err:.3e} > {tol:.3e}"
        f = np.isfinite(wl)
        bits = 2.0 ** -11 if self.typ == "bf16" and magnitude is None else 2.0 ** -19
        assert float(np.abs(e[f] - wl[f]).max(initial=0)) <= top * bits + 1e-6
        return got


# ---- the units that follow the value scales -----------------------------------

@pytest.mark.parametrize("typ,tokens", [("fp32", 1), ("fp16", 1), ("bf16", 1), ("bf16", 4)])
def test_scales_that_rise_after_a_nan(typ, tokens):
    """A NaN group among values of scale 0, then scales above 4 under falling scores: a warp's unit
    follows the scales that come, not the NaN's bits."""
    rng = np.random.default_rng(41)
    batch, heads, group, dim, n = 76, 8, 4, 128, 1024
    unit = np.where(rng.standard_normal(dim) > 0, 1.0, -1.0)
    k, v, q = [], [], []
    for _ in range(batch):
        k.append(np.where(np.arange(n) < 256, 1.0, 0.9)[:, None, None] * unit * np.ones((1, heads, 1)))
        x = np.full((n, heads, dim), 0.5)
        x[8:256:16, :, 40] = x[9:256:16, :, 40] = np.nan   # (an even and an odd key of every tile)
        x[256:] = 100 * rng.standard_normal((n - 256, heads, dim))
        v.append(x)
        q.append(0.2 * unit + 0.01 * rng.standard_normal((tokens, heads * group, dim)))
    s = Given(k, v, q, 64, typ)
    got = s.check(group=32)
    nan = torch.isnan(got)
    assert bool(nan[..., 32:64].all()) and not bool(nan[..., :32].any()) and not bool(nan[..., 64:].any())


# ---- small probabilities --------------------------------------------------------

def sinks(rng, n, heads, dim, at, score):
    """Keys [n, heads, dim] of which those at `at` score `score` (natural units) for queries near
    half the returned direction, and values, large ones, that are 0 at those keys."""
    unit = np.where(rng.standard_normal(dim) > 0, 1.0, -1.0)
    k = rng.standard_normal((n, heads, dim))
    v = 1000 * rng.standard_normal((n, heads, dim))
    k[at] = score / (dim ** -0.5 * 0.5 * dim) * unit
    v[at] = 0
    return k, v, unit


def near(rng, unit, tokens, q_heads):
    return 0.5 * unit + 0.02 * rng.standard_normal((tokens, q_heads, len(unit)))


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("tokens,q_heads", [(1, 4), (3, 8), (40, 4)])
def test_rows_that_a_few_keys_dominate(typ, dim, tokens, q_heads):
    """A key of every 16 takes nearly all of a row and its value is 0: what the others bring is all of
    the result, each at a millionth of the largest probability."""
    rng = np.random.default_rng(42)
    k, v, unit = sinks(rng, 4097, 2, dim, np.s_[3::16], 14.0)
    s = Given([k], [v], [near(rng, unit, tokens, q_heads)], 64, typ)
    s.check(many=tokens * q_heads // 2 > 24)


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("weight", [0.9, 0.99])
@pytest.mark.parametrize("tokens,batch,n", [(1, 38, 4097), (1, 38, 32768), (30, 19, 8192)])
def test_rows_that_one_key_dominates(typ, weight, tokens, batch, n):
    """The first keys (one for every warp that may share an item) have `weight` of each row between
    them and values of 0, under enough sequences that an item is not cut; the sequences share pages."""
    rng = np.random.default_rng(43)
    score = np.log(n * weight / (1 - weight) / 8)
    k, v, unit = sinks(rng, n, 8, 128, np.arange(8) * 16 + 5, score)
    q = [near(rng, unit, tokens, 16) for _ in range(batch)]
    s = Given([k] * batch, [v] * batch, q, 64, typ)
    s.check(many=tokens > 1)


@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("tokens,q_heads", [(1, 4), (3, 8), (40, 4)])
def test_value_groups_of_very_different_scales(typ, tokens, q_heads):
    """Groups of a head at 3000, 1 and 0.02: each is as near as if it were alone."""
    rng = np.random.default_rng(44)
    n, dim = 1000, 128
    k, v = rng.standard_normal((n, 2, dim)), rng.standard_normal((n, 2, dim))
    v[..., :32] *= 3000
    v[..., 64:96] *= 0.02
    s = Given([k], [v], [0.3 * rng.standard_normal((tokens, q_heads, dim))], 16, typ)
    s.check(many=tokens * q_heads // 2 > 24, group=32)


# ---- scores -----------------------------------------------------------------------

@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("tokens,q_heads", [(1, 4), (4, 8)])
def test_scores_of_large_minimums_that_cancel(typ, dim, tokens, q_heads):
    """Keys whose groups lie at +20 and -20 under queries of equal group sums: the minimums' products
    are far larger than the scores.  Few rows have them in 22 bits in all types (the codes are exact,
    bf16 queries too): scores to 4 A 2^-21, A the largest sum of |q_d k_d| scale."""
    rng = np.random.default_rng(47)
    n = 500
    k, v = 0.3 * rng.standard_normal((n, 2, dim)), rng.standard_normal((n, 2, dim))
    k[..., :32] += 20
    k[..., 32:64] -= 20
    q = rng.standard_normal((tokens, q_heads, dim)) + 1
    q[..., 32:64] = q[..., 31::-1]
    a = float((np.abs(q).max((0, 1)) * np.abs(k).max((0, 1))).sum()) * dim ** -0.5
    Given([k], [v], [q], 16, typ).check(magnitude=a)


# ---- where a NaN goes -------------------------------------------------------------

@pytest.mark.parametrize("typ", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("dim,element", [(64, 40), (96, 70), (96, 5), (128, 127)])
@pytest.mark.parametrize("tokens,q_heads,n", [(1, 4, 300), (5, 4, 300), (70, 4, 300), (90, 8, 200), (70, 2, 5000)])
@pytest.mark.parametrize("window", [0, 37])
def test_a_nan_in_a_value_reaches_its_group_alone(typ, dim, element, tokens, q_heads, n, window):
    """A value's NaN is its group's (32 elements) for the rows that see the key, whichever tile holds
    it; the other elements, and lse, have none of it."""
    rng = np.random.default_rng(45)
    k, v = rng.standard_normal((n, 2, dim)), rng.standard_normal((n, 2, dim))
    q = rng.standard_normal((tokens, q_heads, dim))
    for key in {20, n - tokens - 1, n - tokens // 2 - 1, n - 1}:
        x = v.copy()
        x[key, 1, element] = np.nan
        s = Given([k, k[:60]], [x, v[:60]], [q, q[:1]], 16, typ)
        s.check(window=window, many=tokens * q_heads // 2 > 24)


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens", [2, 70])
def test_nan_in_a_key_and_in_several_values(typ, tokens):
    """A key's NaN is the whole row's and its lse's; several values' NaN are their groups'."""
    rng = np.random.default_rng(46)
    n, dim = 700, 128
    k, v = rng.standard_normal((n, 1, dim)), rng.standard_normal((n, 1, dim))
    v[n - 40, 0, 3] = v[n - 41, 0, 70] = v[n - 1, 0, 100] = v[5, 0, 40] = np.nan
    k[n - 2, 0, 9] = np.nan
    Given([k], [v], [rng.standard_normal((tokens, 4, dim))], 32, typ).check(many=tokens > 10)


# ---- how many bits bf16 calls have --------------------------------------------------

@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("tokens,q_heads", [(1, 8), (2, 16), (3, 16), (40, 8)])
def test_bf16_operands_hold_their_bits(dim, tokens, q_heads):
    """Before the output's rounding a bf16 call is within 2^-11 (p and p sc to 11 bits each, 2^-12 at
    most), with many rows 3 2^-12 and the scores' 2^-12 S_rms.  The rounding's own error r is known from
    the exact result; independent errors add as squares (2 % for chance): two bits fewer in an operand
    would show."""
    rng = np.random.default_rng(48)
    n, many = 3000, tokens * q_heads // 2 > 24
    k, v = rng.standard_normal((n, 2, dim)), rng.standard_normal((n, 2, dim))
    s = Given([k] * 4, [v] * 4, [rng.standard_normal((tokens, q_heads, dim)) for _ in range(4)], 64, "bf16")
    got, _ = s.run()
    torch.cuda.synchronize()
    want = s.expect()[0]
    norm = np.linalg.norm(want)
    err = np.linalg.norm(got.double().cpu().numpy() - want) / norm
    r = np.linalg.norm(torch.from_numpy(want).to(torch.bfloat16).double().numpy() - want) / norm
    own = 4 * 2.0 ** -12 if many else 2.0 ** -11   # (S_rms is 1 here)
    assert err <= 1.02 * np.hypot(r, own), f"{err:.3e}, rounding alone {r:.3e}"
