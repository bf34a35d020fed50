"""Lengths far out of range in device memory: moves stay within the table, and the status word says so."""
import pytest
import torch

from test_drafts import cache, ints

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [-2 ** 31, -2 ** 31 + 7, -1, 0, 7, 33, 2 ** 31 - 1])
def test_no_move_by_a_length_out_of_range(length):
    """Eight nodes of a request with room for 32 tokens; the difference of length and nodes may not fit 32 bits."""
    c = cache(5, [8, 6], [10, 5], 2, 2, 64)
    path = ints([0, 3, 6, 7, -1, -1, -1, -1] + [0, -1, -1, -1, -1, -1])
    c["lens"][0] = length
    k, v = (c[n].cuda().view(torch.bfloat16) for n in "kv")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ta.keep_drafts(path.cuda(), ints([0, 8, 14]).cuda(), c["table"].cuda(), c["lens"].cuda(), k, v, status=status)
    assert status.item() == _abi.BATCH_BAD_INPUT
    assert torch.equal(k.view(torch.int16).cpu(), c["k"]) and torch.equal(v.view(torch.int16).cpu(), c["v"])
