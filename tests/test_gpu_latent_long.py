"""Latent attention over long sequences with several row tiles: segments of more pieces than a warp joins, beside
shorter ones.  Random rows against the oracle, and rows that count the tokens of every 16-token block."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gpu_helpers import dev_bf16, dev_i32  # noqa: E402
from test_gpu_latent import check, make, run, values  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402
from gqa_split_kv_gb300.workloads import f32_to_bf16_bits  # noqa: E402

CASES = [(512, 128, 1, [4096]), (512, 128, 1, [20001]), (512, 64, 3, [20001, 17, 4096]), (128, 128, 1, [9000, 20001, 5000, 0, 33]),
         (256, 100, 2, [4096, 4095]), (512, 16, 1, [20001])]


@pytest.mark.parametrize("R,H,q_len,lens", CASES)
def test_matches_oracle(R, H, q_len, lens):
    c = make(H + sum(lens), lens, q_len, H, R, max(lens))
    first = run(c)
    check(first, c, f"R={R} H={H} q_len={q_len} {lens}")
    assert np.array_equal(run(c), first)
    assert binding.device_error() == 0


@pytest.mark.parametrize("ps", [0, 16, 64])
@pytest.mark.parametrize("R,H,q_len,lens", CASES + [(512, 64, 16, [3001, 20001]), (512, 256, 1, [2048, 1, 2047])])
def test_every_block_of_tokens_counts_once(R, H, q_len, lens, ps):
    """Scale 0 weighs every token alike and block t // 16 has a one at latent coordinate (t // 16) % R, so coordinate r of
    the output is the number of visible tokens of its blocks over the number of all: weights, sums and factors are
    exact, the quotient is off by two roundings of fp32 and one of bf16.  At most ten blocks share a coordinate, so one
    lost or taken twice changes it by a tenth at least."""
    top = max(lens)
    c = make(1, [top] * len(lens), q_len, H, R, top, ps)
    t = np.arange(top)
    row = np.zeros((top, R + 64), np.float32)
    row[t, (t // 16) % R] = 1.0
    bits = f32_to_bf16_bits(row)
    if ps:
        for b in range(len(lens)):
            for j in range(-(-top // ps)):
                n = min(ps, top - j * ps)
                c["pool"][c["table"][b, j], :n] = bits[j * ps:j * ps + n]
    else:
        c["rows"][:] = bits
    c["scale"], c["lens"] = 0.0, np.asarray(lens, np.int32)
    got = values(run(c))
    assert -(-top // 16) <= 10 * R
    for b, L in enumerate(lens):
        for i in range(q_len):
            seen = L - q_len + 1 + i
            want = np.bincount((t[:max(seen, 0)] // 16) % R, minlength=R) / max(seen, 1)
            assert np.all(np.abs(got[b, i] - want) <= want * (2.0 ** -8 + 2.0 ** -22)), (b, L, i)
    assert binding.device_error() == 0


def test_a_workspace_of_its_own_size_holds_the_pieces():
    """Bytes behind the workspace stay as they are, with as many pieces as the longest segments have."""
    c = make(3, [20001, 4096], 1, 128, 512, 20001)
    size = binding.latent_workspace(2, 128, 512).numel()
    room = torch.full((size + 4096,), 0x5A, device="cuda", dtype=torch.uint8)
    out = torch.empty(2, 1, 128, 512, device="cuda", dtype=torch.bfloat16)
    binding.latent_attn_contig(dev_bf16(c["q"]), dev_bf16(c["rows"]), dev_i32(c["lens"]), scale=c["scale"],
                               workspace=room[:size], out=out)
    assert bool((room[size:] == 0x5A).all())
    assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), run(c))
