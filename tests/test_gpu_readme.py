"""The readme's Python lines for the cache, run as they stand there on a small batch."""
import re
from pathlib import Path

import pytest

from decode_gemv_gb300 import lw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if torch.cuda.is_available():
    from kv_plain import DEV, generator, i32, read, relative, scores, slots_of, spans, status


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_the_cache_in_readme(typ):
    """All calls succeed; the attention over at most 64 of 32 pages is that over every kept key, within twice what
    lw_kv_attention is held to (fp32 7.6e-5, bf16 1e-2 + 2^-8)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()
    text = (Path(__file__).resolve().parent.parent / "README.md").read_text()
    blocks = [x for x in re.findall(r"```python\n(.*?)```", text, re.S) if "lw_kv_" in x]
    assert len(blocks) == 2
    gen, batch, width, lens = generator(90), 3, 48, [3000, 2049, 100]
    heads, page_table = 8, torch.randperm(3 * 48, device=DEV, generator=gen).to(torch.int32).view(3, 48)

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=gen).to(typ)

    # the prompts, then a step of one token each
    prompt = torch.cat([slots_of(page_table[b], range(n - 1), 64) for b, n in enumerate(lens)])
    names = dict(torch=torch, lw=lw, n_pages=3 * 48, batch=batch, page_table=page_table, st=status(),
                 k=randn(prompt.shape[0], heads, 128), v=randn(prompt.shape[0], heads, 128), slots=prompt,
                 q=randn(batch, 32, 128), out=torch.zeros(batch, 32, 128, dtype=typ, device=DEV),
                 q_start=i32([0, 1, 2, 3]), kv_len=i32([n - 1 for n in lens]))
    exec(blocks[0], names)
    names.update(k=randn(batch, heads, 128), v=randn(batch, heads, 128), kv_len=i32(lens), new_len=i32([0] * batch),
                 slots=torch.cat([slots_of(page_table[b], [n - 1], 64) for b, n in enumerate(lens)]),
                 positions=torch.tensor([n - 1 for n in lens], device=DEV),
                 lse=torch.zeros(batch, 32, device=DEV), weights=torch.zeros(batch, heads, 48 * 64, device=DEV),
                 kept=torch.zeros(batch, heads, 2048, dtype=torch.int32, device=DEV))
    exec(blocks[1], names)
    torch.cuda.synchronize()
    assert int(names["st"]) == 0
    cache, q, out = names["cache"], names["q"], names["out"]
    assert names["kv_len"].tolist() == [2048, 2048, 100]
    tol = 2 * (7.6e-5 if typ == torch.float32 else 1e-2 + 2.0 ** -8)
    for b, n in enumerate(names["kv_len"].tolist()):
        k, v = read(cache, slots_of(page_table[b], range(n), 64))
        p = scores(q[b:b + 1], k, spans(1, n), 128 ** -0.5)[0].softmax(-1)
        assert relative(out[b], torch.einsum("hj,jhd->hd", p, v.double().repeat_interleave(4, 1))) <= tol
