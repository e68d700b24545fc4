"""Calls whose predecessors in a captured graph are several: a fork over two streams and a join, replayed."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gqa_split_kv_gb300 import binding  # noqa: E402


@pytest.mark.parametrize("tokens", [5, 3000])
def test_fork_and_join(tokens):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    H, D, R, ps = 2, 64, 128, 16
    pages = -(-tokens // ps)
    w, w64 = binding.rope_inv_freq(D), binding.rope_inv_freq(64)
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[None]
    k, v = (torch.zeros(1, tokens, H, D, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    latent = torch.zeros(1, tokens, 1, R + 64, device="cuda", dtype=torch.bfloat16)
    q = torch.randn(1, 1, 8, R + 64, generator=gen, device="cuda").to(torch.bfloat16)
    pos, lens = torch.arange(tokens, device="cuda", dtype=torch.int32)[None], torch.tensor([tokens], device="cuda", dtype=torch.int32)
    pool = [torch.zeros(pages, ps, H, D, dtype=torch.int8, device="cuda") for _ in "kv"]
    scale = [torch.zeros(pages, H, ps, device="cuda") for _ in "kv"]
    rows = torch.zeros(pages, ps, R + 64, dtype=torch.bfloat16, device="cuda")
    x, back = torch.empty_like(k), [torch.empty_like(k) for _ in "kv"]
    out, y = torch.empty(1, 1, 8, R, device="cuda", dtype=torch.bfloat16), torch.empty_like(k)
    side = torch.cuda.Stream()

    def step(fork):
        main = torch.cuda.current_stream()
        other = side if fork else main
        other.wait_stream(main)
        binding.rope_apply(k, pos, w, out=x)
        with torch.cuda.stream(other):
            binding.kv_write_paged(latent, None, rows[:, :, None], None, table, lens, tokens, inv_freq=w64, offset=R)
            binding.latent_attn_paged(q, rows, table, lens, tokens, scale=0.1, out=out)
        binding.kv_write_int8_paged(x, v, *pool, *scale, table, lens, tokens)
        main.wait_stream(other)
        binding.kv_read_int8_paged(*pool, *scale, table, lens, tokens, tokens, k_out=back[0], v_out=back[1], zero_rest=True)
        other.wait_stream(main)
        with torch.cuda.stream(other):  # after both branches
            binding.rope_apply(back[0], pos, w, backward=True, out=y)
        main.wait_stream(other)
        y.add_(out.float().mean().to(torch.bfloat16))

    def feed():
        for t in (k, v, latent):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))

    feed()
    step(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(True)
    for _ in range(4):
        feed()
        graph.replay()
        got = [t.clone() for t in (y, out, *back, *pool, *scale, rows)]
        step(False)  # one stream, eager
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, out, *back, *pool, *scale, rows)))
    assert binding.device_error() == 0
