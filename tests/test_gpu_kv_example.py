"""examples/kv_attention_block.py on the GPU: coded projections, the 4-bit
cache and attention together, prompts of different lengths and captured steps,
against a plain computation on the cached values (tolerance: that of the coded
products, 1e-3 of the largest output)."""
import importlib.util
from pathlib import Path

import pytest

from helpers import TOL

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = Path(__file__).resolve().parent.parent / "examples" / "kv_attention_block.py"
    spec = importlib.util.spec_from_file_location("kv_attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("prompts,steps", [((37, 5, 120, 200), 5), ((1,), 3), ((300, 64, 63, 65, 1, 2, 16, 17), 2)])
def test_block(example, prompts, steps):
    r = example.main(prompts, steps)
    assert r["error"] <= TOL, r
    assert r["tokens"] == sum(prompts) + steps * len(prompts)
    assert r["cache_bytes"] * 3 < r["bf16_bytes"]
