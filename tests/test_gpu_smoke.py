"""The smoke run's calls over long caches reach every form that such a call has."""
import os
import re

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import __graft_entry__ as entry  # noqa: E402
from gqa_split_kv_gb300 import binding, build  # noqa: E402


def test_both_forms_of_a_prefix_run(monkeypatch):
    """Rows of a KV head behind the prefix: some calls with few, which seg_kernel takes alone, some with more than it takes."""
    rows, call = [], binding.prefix_attn_contig

    def record(q, k_prefix, *args, **kw):
        rows.append(q.shape[0] * q.shape[1] * q.shape[2] // k_prefix.shape[1])
        return call(q, k_prefix, *args, **kw)

    monkeypatch.setattr(binding, "prefix_attn_contig", record)
    entry.smoke_long_caches(torch.device("cuda:0"))
    with open(os.path.join(build.CSRC, "prefix_attn.cu")) as f:
        few = int(re.search(r"kFewRows = (\d+)", f.read()).group(1))
    assert min(rows) <= few < max(rows)


def test_both_forms_of_weights_run(monkeypatch):
    """One token's rows and a window's."""
    rows, call = [], binding.kv_weights_contig

    def record(q, k, *args, **kw):
        rows.append(q.shape[1] * q.shape[2] // k.shape[2])
        return call(q, k, *args, **kw)

    monkeypatch.setattr(binding, "kv_weights_contig", record)
    entry.smoke_long_caches(torch.device("cuda:0"))
    assert min(rows) <= 16 < max(rows)
