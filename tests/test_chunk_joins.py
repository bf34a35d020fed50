"""Segments of two steps, one behind another: the halves' maxima and sums are exchanged at every segment's end, and
the half that begins the next segment has only that one step there.  The same bits again and again, and the
definition's numbers.  Tolerances: test_chunk_attention.py."""
import pytest
import torch

from test_chunk_attention import attend, check, make, to_gpu

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("trees", [None, "mixed"])
@pytest.mark.parametrize("lens,heads,d", [
    ([129 + i % 128 for i in range(700)], (8, 4), 64),          # two steps, always
    ([129 + i % 128 for i in range(300)], (32, 8), 128),
    ([256, 300, 129, 384, 140] * 100, (8, 2), 128),             # two and three: the halves swap places
    ([128, 200, 60, 250, 256, 257] * 100, (4, 4), 64),          # and one
])
def test_short_segments_in_a_row(lens, heads, d, trees):
    # maxima that differ from segment to segment and from half to half
    new = [1 + i % 3 for i in range(len(lens))]
    s = make(len(lens), lens, new, *heads, d, trees=trees, gain=2.0)
    c = to_gpu(s)
    want = attend(c)
    check(s, *want)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for i in range(200):
        if i % 20 == 0:
            flush.fill_(i)
        out, lse = attend(c)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
