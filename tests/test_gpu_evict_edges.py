"""Eviction at its edges: caches without a token."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import lens_of  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("int8", [False, True])
def test_a_cache_without_a_token(paged, int8):
    """Rows and pages that do not exist: nothing is kept, and the weights of the outputs are zeros."""
    dt = torch.int8 if int8 else torch.bfloat16
    slabs, slab = (0, 16) if paged else (2, 0)
    k, v = (torch.empty(slabs, slab, 3, 32, dtype=dt, device="cuda") for _ in "kv")
    numbers = [torch.empty(slabs, 3, slab, device="cuda") for _ in range(3 if int8 else 1)]
    out = dict(k_out=torch.full((2, 6, 3, 32), 3, device="cuda").to(dt), weights_out=torch.full((2, 3, 6), 5.0, device="cuda"))
    out["v_out"] = out["k_out"].clone()
    if int8:
        out["k_scale_out"], out["v_scale_out"] = (torch.full((2, 3, 6), 5.0, device="cuda") for _ in "kv")
    old = {x: y.clone() for x, y in out.items()}
    pages = (torch.zeros(2, 4, dtype=torch.int32, device="cuda"), lens_of(5, 0), 64) if paged else (lens_of(5, 0),)
    fn = getattr(binding, "kv_evict" + ("_int8" if int8 else "") + ("_paged" if paged else "_contig"))
    kept, new_lens = fn(k, v, *numbers, *pages, 4, **out)
    assert (kept == -1).all() and new_lens.tolist() == [0, 0]
    assert not out["weights_out"].any()
    for x in out:
        if x != "weights_out":
            assert torch.equal(out[x], old[x])
    assert binding.device_error() == 0
