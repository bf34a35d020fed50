"""Attention behind a shared prefix from several streams, graphs and host
threads at once, with the tensor-core tiles: each run has a workspace of its
own, so that all give what one alone gives, bit for bit."""
import pytest
import torch

from test_host_threads import together
from test_prefix_attention import attend, check, make, to_gpu

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu

BATCHES = [
    ([100] * 40, None, (16, 4), 128, 5001),       # tiles beside and behind the own pages
    ([300, 20, 77] * 6, [2, 1, 4] * 6, (16, 2), 64, 1000),
    ([30] * 400, None, (4, 2), 64, 333),          # more than 384 requests: a kernel more
    ([500] * 7, None, (4, 4), 128, 2000),         # the prefix in the line
]


def batch(i):
    lens, new, heads, d, prefix = BATCHES[i]
    s = make(i, lens, new, *heads, d, prefix)
    return s, to_gpu(s)


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_two_streams_and_two_graphs(i):
    s, c = batch(i)
    want = attend(c)
    check(s, *want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    runs = [attend(c, stream=streams[k % 2]) for k in range(20)]
    torch.cuda.synchronize()
    assert all(same(want, r) for r in runs)
    graphs, outs = [], []
    for stream in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(attend(c))
        graphs.append(g)
    for _ in range(10):
        for o in outs:
            o[0].fill_(7), o[1].fill_(7)
        torch.cuda.synchronize()
        for stream, g in zip(streams, graphs):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(want, o) for o in outs)


def test_host_threads_with_other_batches():
    def work_of(i):
        _, c = batch(i)
        want = attend(c)

        def work(k):
            got = attend(c)
            if k % 50 == 49:
                assert same(want, got)
        return work

    together(*(work_of(i) for i in range(len(BATCHES))), calls=400)
