"""Cache reads that write every row of their outputs: zeros where no token lies."""
import numpy as np
import pytest

from oracle import cache_ops as oc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gpu_helpers import dev, dev_i32, host_bits  # noqa: E402
from test_gpu_cache_ops import LENS, to_dev, write_case  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


def read(c, lens, n, starts=None, **kw):
    cache, scale, lens = [to_dev(x) for x in c["cache"]], [dev(x) for x in c["scale"]], dev_i32(np.asarray(lens))
    kw["starts"] = None if starts is None else dev_i32(starts)
    if len(cache) == 1:
        cache.append(None)
    if c["ps"] and c["scale"]:
        return binding.kv_read_int8_paged(*cache, *scale, dev_i32(c["table"]), lens, c["cap"], n, **kw)
    if c["ps"]:
        return binding.kv_read_paged(*cache, dev_i32(c["table"]), lens, c["cap"], n, **kw)
    return binding.kv_read_int8_contig(*cache, *scale, lens, n, **kw)


def want(c, lens, n, starts=None):
    shape = (len(lens), n, c["H"], c["D"])
    return [oc.read(np.zeros(shape, np.uint16), x, lens, c["cap"], n, starts, c["table"], c["ps"],
                    c["scale"][i] if c["scale"] else None) for i, x in enumerate(c["cache"])]


def stale(c, B, n):
    """Outputs that an earlier, unrelated use left full of NaN."""
    return [torch.full((B, n, c["H"], c["D"]), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in "kv"]


@pytest.mark.parametrize("ps,int8", [(0, True), (16, True), (48, True), (16, False), (40, False)])
@pytest.mark.parametrize("H,D", [(8, 128), (1, 576), (3, 32)])
def test_every_row_is_written(ps, int8, H, D):
    c = write_case(D + ps, len(LENS), 1, H, D, LENS, 104, ps, int8)
    rng = np.random.default_rng(ps + 1)
    for starts, n in ((None, 104), (rng.integers(-30, 90, len(LENS)).astype(np.int32), 41), (None, 1)):
        ref = want(c, LENS, n, starts)
        out = stale(c, len(LENS), n)
        read(c, LENS, n, starts, k_out=out[0], v_out=out[1], zero_rest=True)
        made = read(c, LENS, n, starts)
        one = stale(c, len(LENS), n)[0]
        one.zero_()
        mixed = read(c, LENS, n, starts, k_out=one)  # the one made here is filled, the given one is left
        for i in range(2):
            assert np.array_equal(host_bits(out[i]), ref[i])
            assert np.array_equal(host_bits(made[i]), ref[i]) and np.array_equal(host_bits(mixed[i]), ref[i])
    assert binding.device_error() == 0


def test_a_long_call_then_a_shorter_one_into_the_same_outputs():
    c = write_case(5, 3, 1, 2, 64, [90, 64, 33], 96, 16, True)
    out = stale(c, 3, 96)
    for lens in ([90, 64, 33], [10, 0, 33], [0, 0, 0], [1, 96, 2]):
        c["lens"] = np.asarray(lens, np.int32)
        c["table"] = np.arange(18, dtype=np.int32).reshape(3, 6) % len(c["cache"][0])
        read(c, lens, 96, k_out=out[0], v_out=out[1], zero_rest=True)
        for i, ref in enumerate(want(c, lens, 96)):
            assert np.array_equal(host_bits(out[i]), ref)
    assert binding.device_error() == 0


def test_bad_pages_empty_caches_and_keys_only():
    c = write_case(2, 2, 1, 2, 64, [40, 33], 48, 16, True)
    c["table"][0, 1], c["table"][1, 2] = 999, -7
    out = stale(c, 2, 48)
    read(c, c["lens"], 48, k_out=out[0], v_out=out[1], zero_rest=True)
    for i, ref in enumerate(want(c, c["lens"], 48)):
        assert np.array_equal(host_bits(out[i]), ref)
    assert binding.device_error() == 4
    c = write_case(3, 2, 1, 1, 576, [20, 7], 32, 16, False, keys_only=True)
    k, v = read(c, c["lens"], 32, k_out=stale(c, 2, 32)[0], zero_rest=True)
    assert v is None and np.array_equal(host_bits(k), want(c, c["lens"], 32)[0])
    pool = torch.zeros(0, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
    table, out = torch.zeros(2, 3, device="cuda", dtype=torch.int32), [torch.ones(2, 4, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    binding.kv_read_paged(pool, pool.clone(), table, dev_i32(np.array([5, 0])), 48, 4, k_out=out[0], v_out=out[1],
                          zero_rest=True)
    assert not out[0].any() and not out[1].any()
    assert binding.device_error() == 0
