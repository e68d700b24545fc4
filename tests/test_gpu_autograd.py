"""Beside autograd: the calls are not recorded, and what they write is known to have changed."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gqa_split_kv_gb300 import binding  # noqa: E402


def randn(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(len(shape)), device="cuda", dtype=dtype)


def test_a_saved_tensor_rotated_in_place_is_noticed():
    x = randn(4, 2, 64, dtype=torch.float32).requires_grad_()
    y = x * 2
    z = (y * y).sum()  # saves y
    pos, w = torch.arange(4, device="cuda", dtype=torch.int32), binding.rope_inv_freq(64)
    with torch.no_grad():
        binding.rope_apply(y, pos, w, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    with pytest.raises(ValueError, match="gradient"):
        binding.rope_apply(x, pos, w, out=x)
    assert not binding.rope_apply(x, pos, w).requires_grad


def test_every_given_output_counts_as_changed():
    lens = torch.tensor([5, 3], device="cuda", dtype=torch.int32)
    k, v = (torch.zeros(2, 8, 2, 64, device="cuda", dtype=torch.int8) for _ in "kv")
    ks, vs = (torch.zeros(2, 2, 8, device="cuda") for _ in "kv")
    ko, vo = randn(2, 8, 2, 64), randn(2, 8, 2, 64)
    new = randn(2, 3, 2, 64)
    o1, o2 = randn(2, 1, 4, 128), randn(2, 3, 4, 64)
    kv = randn(2, 8, 4, 128)

    def calls():
        binding.kv_write_int8_contig(new, new.clone(), k, v, ks, vs, lens)
        binding.kv_read_int8_contig(k, v, ks, vs, lens, 8, k_out=ko, v_out=vo)
        binding.latent_attn_contig(randn(2, 1, 4, 192), randn(2, 8, 192), lens, scale=0.1, out=o1)
        binding.latent_prefill_contig(randn(2, 3, 4, 128), kv[..., :64], randn(2, 8, 64), kv[..., 64:], lens, scale=0.1,
                                      out=o2)

    outs = (k, v, ks, vs, ko, vo, o1, o2)
    before, inputs = [t._version for t in outs], [t._version for t in (new, lens, kv)]
    calls()
    assert all(t._version > b for t, b in zip(outs, before))
    assert [t._version for t in (new, lens, kv)] == inputs
    want = [t.clone() for t in outs]
    with torch.inference_mode():  # inference tensors have no version
        k, v, ks, vs, ko, vo, o1, o2 = outs = [t.clone() for t in outs]
        calls()
    calls()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert binding.device_error() == 0
