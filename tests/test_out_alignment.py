"""Outputs of a plan's run that lie 16 but not 32 bytes past a boundary, as the header allows: the same bits as
elsewhere, and nothing written beside them."""
import pytest
import torch

import workloads as W
from parity_utils import compare, make_inputs, oracle_on_tokens

pytestmark = pytest.mark.gpu

GUARD = 12345.0


@pytest.mark.parametrize("off", [4, 8])  # floats
@pytest.mark.parametrize("options", [{}, {"force_path": 1}, {"force_path": 2}, {"split_tokens": 64},
                                     {"split_tokens": 64, "merge_mode": 1}, {"force_path": 2, "split_tokens": 128}])
@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (32, 2, 64)])
def test_half_a_sector_off(hq, hkv, d, options, off):
    import tree_structured_decode_gb300 as ta

    spec = W.random_tree(11, n_nodes=20, max_len=300, hq=hq, hkv=hkv, d=d, zero_len_prob=0.1, max_queries_per_node=4)
    q, k, v = make_inputs(spec, tail_fill=float("nan"))
    n = spec.n_queries * hq * d
    with ta.Plan.from_spec(spec, **options) as p:
        want, want_lse = p.run(q, k, v)
        room = torch.full((n + 16,), GUARD, device="cuda")
        out = room[off: off + n].view(spec.n_queries, hq, d)
        assert out.data_ptr() % 32 == 4 * off % 32
        lse = torch.empty_like(want_lse)
        p.run(q, k, v, out=out, lse=lse)
        torch.cuda.synchronize()
        assert p.device_status() == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert (room[:off] == GUARD).all() and (room[off + n:] == GUARD).all()
        room.fill_(GUARD)
        assert p.run_static(q, k, v, out, lse) == 0
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert (room[:off] == GUARD).all() and (room[off + n:] == GUARD).all()
    ref, ref_lse = oracle_on_tokens(spec, q, k, v, list(range(spec.n_queries)))
    compare(out, lse, ref, ref_lse)
