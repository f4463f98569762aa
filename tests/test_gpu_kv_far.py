"""The calls around the 4-bit cache where addresses pass 2^31: the answer does not depend on where the pages, the
weights' rows or the summaries lie, so every result is the small pool's, bit for bit."""
import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from kv_plain import DEV, generator, i32, read, slots_of, status


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


def run(cache, table, out_table, weights, heads, dim, page, lens):
    """Two sequences written with rotary positions, weighed by few rows and by many, sparsely attended to, and cut
    down into other pages and in place: all results."""
    gen, st, group, tokens = generator(70), status(), 2, 100
    n, width = i32(lens), table.shape[1]
    angles = torch.empty(1000, dim, device=DEV)
    lw.lw_rotary_table(angles)
    for b, length in enumerate(lens):
        k, v = (torch.randn(length, heads, dim, device=DEV, generator=gen) for _ in range(2))
        pos = torch.arange(length, device=DEV)
        lw.lw_kv_write_rotary(cache, k, v, slots_of(table[b], range(length), page), pos, angles, st)
    summary = torch.empty(lw.lw_kv_summary_bytes(cache), dtype=torch.uint8, device=DEV)
    lw.lw_kv_summarise(cache, summary, i32([0, 0]), n, table, st)
    got = []
    for T in (1, tokens):
        q = torch.randn(2 * T, heads * group, dim, device=DEV, generator=gen).to(torch.bfloat16)
        start, out, lse = i32([0, T, 2 * T]), torch.empty_like(q), torch.empty(2 * T, heads * group, device=DEV)
        chosen = torch.empty(2 * T, heads, 4, dtype=torch.int32, device=DEV)
        ws = torch.zeros(max(lw.lw_kv_workspace_bytes(cache, heads * group, 2 * T, 2),
                             lw.lw_kv_weigh_workspace_bytes(cache, heads * group, 2 * T),
                             lw.lw_kv_blocks_workspace_bytes(cache, heads * group, 2 * T, width, 4)), dtype=torch.uint8,
                         device=DEV)
        lw.lw_kv_attention(cache, q, start, n, table, out, ws, st, max_q=T, lse=lse)
        lw.lw_kv_weigh(cache, q, lse, start, n, table, weights, ws, st, max_q=T, add_to=weights if T > 1 else None)
        got += [out.clone(), lse, *(weights[b, :, :x].clone() for b, x in enumerate(lens))]
        lw.lw_kv_attention_blocks(cache, summary, q, start, n, table, out, ws, st, blocks=4, chosen=chosen)
        got += [out, chosen]
    kept, out_len = torch.empty(2, heads, 50, dtype=torch.int32, device=DEV), i32([0, 0])
    for to in (out_table, table):
        lw.lw_kv_evict(cache, weights, n, table, to, out_len, weights if to is table else None, kept, st, keep=50,
                       first=1, recent=9)
        got += [kept.clone(), out_len.clone()]
        for b in range(2):
            got += list(read(cache, slots_of(to[b], range(50), page)))
    got += [weights[b, :, :x].clone() for b, x in enumerate(lens)]
    torch.cuda.synchronize()
    assert int(st) == 0
    return got


@pytest.mark.parametrize("heads,dim,page,pages", [(8, 128, 64, 30000), (1, 64, 16, 15200000)])
def test_far_addresses(heads, dim, page, pages):
    """A pool past 2^31 bytes (the second one's summaries too), weights whose sequences lie 2^31 elements apart."""
    lens, width = [300, 170], -(-300 // page)
    size = lw.lw_kv_page_bytes(heads, dim, page)
    results = []
    for count in (4 * width, pages):
        ids = torch.randperm(4 * width, device=DEV, generator=generator(71)).to(torch.int32) + (count - 4 * width)
        cache = lw.KvCache(torch.empty(count * size, dtype=torch.uint8, device=DEV), heads, dim, page)
        far = count == pages
        assert not far or (count - 4 * width) * size > 2 ** 31
        assert not far or dim == 128 or (count - 4 * width) * (2 * dim + 16) > 2 ** 31
        apart = 2 ** 31 + 5 if far else heads * 310
        store = torch.empty(apart + heads * 310, device=DEV)
        weights = store.as_strided((2, heads, 300), (apart, 310, 1))
        ids = ids.view(4, width)
        results.append(run(cache, ids[:2].contiguous(), ids[2:].contiguous(), weights, heads, dim, page, lens))
        del cache, store, weights
        torch.cuda.empty_cache()
    for x, y in zip(*results):
        assert x.shape == y.shape and torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
