"""Which keys a row sees, key by key, behind long contexts and in large pools.

All keys are zero, so every key that is seen has the same weight, 1, and the sum of
weights is their number n, exactly.  Column c of V is 1024 at one key and 0 at the
others: the output is 1024 / n where the row sees that key and 0 where it does not,
rounded once; a key that is lost, read twice or seen by mistake shows, and so does a
wrong n.  lse = ln n: its logarithm is off by 2^-22 of itself at most."""
import math

import numpy as np
import pytest
import torch

from oracle import drafts as oracle
from test_chunk_attention import attend, make, to_gpu

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


def planted(s, offset, d):
    """Positions of the planted keys of each request, spread over it from `offset`."""
    s["k"][:], s["v"][:] = 0, 0
    where = []
    for b, length in enumerate(s["lens"].tolist()):
        at = (offset + np.arange(d) * max(1, length // d)) % length
        where.append(at)
        for c, x in enumerate(at):
            s["v"][s["table"][b, x // 16], :, x % 16, c] = 1024
    return where


def check_planted(s, where, out, lse):
    out, lse, half = out.double().cpu().numpy(), lse.double().cpu().numpy(), 2.0 ** -8
    for b, length in enumerate(s["lens"].tolist()):
        first, n = int(s["cu_all"][b]), int(s["cu_all"][b + 1] - s["cu_all"][b])
        above = None if s["parents"] is None else oracle.ancestors(s["parents"][first:first + n].tolist())
        for i in range(n):
            if above is None:
                seen = where[b] < length - n + i + 1
                count = length - n + i + 1
            else:
                seen = (where[b] < length - n) | np.isin(where[b] - (length - n), above[i])
                count = length - n + len(above[i])
            want = np.where(seen, 1024 / count, 0)
            assert (np.abs(out[first + i] - want) <= half * want).all(), (b, i)
            assert np.abs(lse[first + i] - math.log(count)).max() <= 2.0 ** -21 * (1 + math.log(count))


@pytest.mark.parametrize("offset", [0, 7, 63])
@pytest.mark.parametrize("lens,new,heads,d,trees", [
    ([5003, 1291], [64, 3], (8, 2), 128, "mixed"), ([700, 2050, 129], [700, 40, 129], (4, 1), 64, None),
    ([9000], [1], (1, 1), 128, None), ([33000], [17], (16, 1), 64, "star"), ([3000], [1500], (5, 1), 64, None),
    ([128 * 40 + 1] * 3, [127, 128, 2], (2, 2), 64, "mixed")])
def test_every_key_counts_once(lens, new, heads, d, trees, offset):
    s = make(offset, lens, new, *heads, d, trees=trees)
    where = planted(s, offset, d)
    out, lse = attend(to_gpu(s))
    check_planted(s, where, out, lse)


def test_pools_past_32_bits():
    """Pools of more than 2^31 elements whose last pages are used: attention, and the move of drafts."""
    pages, hkv, d = 2 ** 31 // (8 * 16 * 128) + 500, 8, 128
    s = make(1, [300, 40], [30, 40], 8, hkv, d, trees="mixed")
    where = planted(s, 3, d)
    c = to_gpu(s)
    k = torch.zeros((pages, hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((pages, hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    last = pages - len(c["v"])
    v[last:] = c["v"]
    c.update(k=k, v=v, table=torch.where(c["table"] >= 0, c["table"] + last, c["table"]))
    out, lse = attend(c)
    check_planted(s, where, out, lse)
    path = torch.tensor([0, 5, 9] + [-1] * 27 + [0, 39] + [-1] * 38, dtype=torch.int32, device="cuda")
    ta.keep_drafts(path, c["cu"], c["table"], c["lens"], k, v)
    want = oracle.keep_drafts(path.tolist(), s["cu_all"], s["table"].numpy(), s["lens"].numpy(),
                              s["k"].float().numpy()[None], s["v"].float().numpy()[None])
    assert np.array_equal(v[last:].float().cpu().numpy(), want[1][0]) and not v[:last].any()


def test_scores_past_32_bits():
    """Rows whose logits begin more than 2^31 elements behind the first's."""
    rows, vocab = 17000, 128000
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(vocab, device="cuda")
    tokens = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    got = ta.token_logprobs(x, tokens, top=3)
    alone = ta.token_logprobs(x[-1:], tokens[-1:], top=3)
    assert got[2][-1].tolist() == alone[2][0].tolist()
    for a, b in zip(got, alone):
        assert torch.allclose(a[-1].float(), b[0].float(), rtol=1e-6, atol=1e-6)
    assert got[2][0].tolist() == [0, 1, 2] and abs(got[1][0].item() - math.log(vocab)) < 1e-5
