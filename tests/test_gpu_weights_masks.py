"""Attention weights over lengths whose products pass 32 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gqa_split_kv_gb300 import binding  # noqa: E402


def test_lengths_whose_products_with_the_group_pass_32_bits():
    """One new token of 64 heads over 34 million equal keys: every weight is 64 / L.  The sums of a CTA's range are whole
    numbers below 2^24, joining 304 of them rounds by 2^-24 each, and so do 64 additions and the reciprocal."""
    L, G, D = 34_000_000, 64, 64
    k = torch.zeros(1, L, 1, D, dtype=torch.int8, device="cuda")
    scale = torch.ones(1, 1, L, device="cuda")
    q = torch.randn(1, 1, G, D, device="cuda").to(torch.bfloat16)
    w = binding.kv_weights_int8_contig(q, k, scale, None)
    off = (w.double() * (L / G) - 1).abs().max().item()
    assert off <= 400 * 2.0 ** -24, off
    assert binding.device_error() == 0
