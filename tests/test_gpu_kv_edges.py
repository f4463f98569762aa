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
