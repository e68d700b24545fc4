"""Rotary positions in a cache that is cut to a budget: places are no longer positions."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import check_attention, f64, lens_of, randn, score_error  # noqa: E402
from oracle import cache_ops as oc  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


def near_rotated(row, k, position, w):
    """One rounding to bf16 (2^-8 of it) of a rotation in fp32 (2^-22 of the head's length, angles exact to 2e-7)."""
    want = oc.rotate(k, position, w)
    return (np.abs(row - want) <= 2.0 ** -8 * np.abs(want) + 2e-6 * np.linalg.norm(k)).all()


def test_steps_with_positions_of_the_programs_own():
    B, Hq, Hkv, D, cap, budget, keep = 2, 8, 2, 64, 128, 60, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = binding.rope_inv_freq(D)
    freq = w.cpu().numpy()
    k, v = (torch.zeros(B, cap, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    weights = torch.zeros(B, Hkv, cap, device="cuda")
    seq, position = lens_of(0, 0), torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    held = [[[] for _ in range(Hkv)] for _ in range(B)]  # (key before its rotation, position) of every place
    cuts = 0
    for step in range(100):
        new_k, new_v, q = randn(gen, B, 1, Hkv, D), randn(gen, B, 1, Hkv, D), randn(gen, B, 1, Hq, D)
        seq += 1
        binding.kv_write_contig(binding.rope_apply(new_k, position, w), new_v, k, v, seq)
        q = binding.rope_apply(q, position, w)
        out = binding.decode_attn_contig(q[:, 0].contiguous(), k, v, seq)
        binding.kv_weights_contig(q, k, weights, seq)
        L = int(seq[0])
        for b in range(B):
            for h in range(Hkv):
                held[b][h].append((f64(new_k[b, 0, h]), step))
                if step % 7 == 0 or step == 99:
                    rows, heads = f64(k[b, :L, h]), slice(h * 4, h * 4 + 4)
                    assert all(near_rotated(r, x, t, freq) for r, (x, t) in zip(rows, held[b][h]))
                    want, mass = ol.attend(f64(q[b])[:, heads], rows[:, None], f64(v[b, :L, h])[:, None], D ** -0.5)
                    check_attention(f64(out[b:b + 1, heads]), want, mass, score_error(f64(q[b]), rows, D ** -0.5, D))
        position += 1
        if L > budget:
            cuts += 1
            kept, new_lens = binding.kv_evict_contig(k, v, weights, seq, keep, first=4, recent=16)
            seq.copy_(new_lens)
            at = kept.cpu().numpy()
            held = [[[held[b][h][i] for i in at[b, h]] for h in range(Hkv)] for b in range(B)]
    assert cuts == 2 and len({tuple(t for _, t in held[0][h]) for h in range(Hkv)}) == Hkv  # heads keep their own
    assert binding.device_error() == 0


def test_a_write_with_frequencies_rotates_by_the_place():
    D = 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    w = binding.rope_inv_freq(D)
    k, v = (randn(gen, 1, 100, 1, D) for _ in "kv")
    _, new_lens = binding.kv_evict_contig(k, v, torch.rand(1, 1, 100, device="cuda", generator=gen), lens_of(90), 30)
    new = randn(gen, 1, 1, 1, D)
    seq = new_lens + 1
    binding.kv_write_contig(new, new, k, v, seq, w)
    assert near_rotated(f64(k[0, 30, 0]), f64(new[0, 0, 0]), 30, w.cpu().numpy())
