"""Where the 4-bit cache's attention can go wrong on the GPU, beyond lengths and
masks: the copies' ring places under long axes, and arguments that the work
queued just before the call writes."""
import pytest

from decode_gemv_gb300 import lw
from test_gpu_kv import DEV, Setup

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lw.load()


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_ring_places_are_reused(typ, tokens, dim):
    """Few rows on long axes: each place of a warp's ring is read and refilled many times, within an
    item and by the next one.  Right, and the same bits call after call."""
    s = Setup(31, [tokens] * 6, [9000, 1, 3000, 0, 2500, 4097], 8, 2, dim, 16, typ)
    first = s.check()
    for _ in range(20):
        again, _ = s.run()
        assert torch.equal(again, first)


@pytest.mark.parametrize("typ,q_len", [("bf16", [1, 1, 1]), ("fp32", [40, 33, 64])])
def test_arguments_written_just_before_the_call(typ, q_len):
    """Lengths, query ranges and the page table come from the work in front of the call, step after
    step of one captured graph."""
    s = Setup(32, q_len, [130, 64, 70], 8, 2, 128, 16, typ)
    want, _ = s.run(lse=False)
    fresh = [t.clone() for t in (s.lens, s.start, s.table)]
    out = torch.zeros_like(want)
    ws = torch.zeros(lw.lw_kv_workspace_bytes(s.cache, 8, sum(q_len), 3), dtype=torch.uint8, device=DEV)
    token = torch.zeros(1, 2, 128, device=DEV)
    none = torch.full((1,), -1, dtype=torch.int64, device=DEV)
    g = lw.StepGraph(torch.cuda.Stream())
    with g.capture():
        for t, f in zip((s.lens, s.start, s.table), fresh):
            t.copy_(f)
        lw.lw_kv_write(s.cache, token, token, none, s.st)   # (a call that lets the next one start early)
        s.run(lse=False, out=out, ws=ws)
        s.lens.fill_(1)          # what a stale read would find
        s.start.fill_(0)
        s.table.fill_(-1)
    for _ in range(5):
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.launch()
        torch.cuda.synchronize()
        assert int(s.st) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("typ", ["fp32", "bf16"])
@pytest.mark.parametrize("hint", [1, 3, 1000])
def test_a_small_calls_workspace_is_enough(typ, hint):
    """Few rows in all, whatever max_q says: right on the workspace asked for, and nothing behind it is
    written."""
    s = Setup(33, [2, 0, 3, 1], [3000, 5, 700, 0], 8, 2, 128, 16, typ)
    need = lw.lw_kv_workspace_bytes(s.cache, 8, 6, 4)
    assert need < lw.lw_kv_workspace_bytes(s.cache, 8, 7, 4)
    room = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device=DEV)
    room[:need] = 0
    s.check(max_q=hint, ws=room[:need])
    assert bool((room[need:] == 0x5A).all())
