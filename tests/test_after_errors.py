"""A call that fails on the host leaves nothing behind that fails the next one."""
import pytest
import torch

import workloads as W

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


def too_large_a_plan():
    """A plan whose partial results need more memory than any GPU has here: refused by the allocation."""
    spec = W.two_level(100000, 16000, 16, 128, 1, 128, seed=1)
    with pytest.raises(ta.TreeAttnError, match="TA_ERR_OOM"):
        ta.Plan.from_spec(spec, split_tokens=128, min_split_tokens=128, split_waves=10000).close()


def test_an_append_after_a_plan_that_was_too_large():
    k, v = (torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    new = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([1, 17, 30], dtype=torch.int32, device="cuda")
    spec = W.config_tiny()
    with ta.Plan.from_spec(spec) as plan:
        _, pk, pv = W.make_tensors(spec, device="cuda:0")
        rows = torch.zeros((spec.n_queries, spec.n_kv_heads, spec.head_dim), dtype=torch.bfloat16, device="cuda")
        too_large_a_plan()
        ta.append_slots(new, new, slots, k, v)
        too_large_a_plan()
        plan.append_kv(rows, rows, pk, pv)
    assert k.sum().item() == v.sum().item() == 3 * 64


def test_many_requests_after_a_plan_that_was_too_large():
    """More than 384 requests: another kernel sums them up."""
    requests = 400
    q = torch.ones((requests, 1, 64), dtype=torch.bfloat16, device="cuda")
    pool = torch.ones((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((requests, 1), dtype=torch.int32, device="cuda")
    lens = torch.full((requests,), 5, dtype=torch.int32, device="cuda")
    too_large_a_plan()
    out, _ = ta.prefix_attention(q, pool, pool, table, lens)
    assert (out == 1).all()
