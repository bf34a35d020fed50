"""Attention of prompts and trees from several streams, graphs and host threads at
once: each run has a workspace of its own, so that all give what one alone gives,
bit for bit."""
import pytest
import torch

from test_chunk_attention import attend, check, make, to_gpu
from test_host_threads import together

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu

BATCHES = [
    ([900, 77, 1500], [900, 77, 1500], (16, 2), 128, None),   # prompts: two tiles a block
    ([3000, 500, 20, 6000] * 4, [26, 9, 20, 1] * 4, (8, 2), 128, "mixed"),
    ([60] * 400, [3] * 400, (4, 2), 64, "star"),              # segments of one step, many requests
    ([9000], [100], (4, 1), 64, "mixed"),                     # one segment, all over the GPU
]


def batch(i):
    lens, new, heads, d, trees = BATCHES[i]
    s = make(i, lens, new, *heads, d, trees=trees, padding=2)
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
        want, got = attend(c), [None]

        def work(k):
            got[0] = attend(c)
            if k % 100 == 99:
                torch.cuda.current_stream().synchronize()
                assert same(want, got[0])
        return work

    together(*(work_of(i) for i in range(len(BATCHES))), calls=400)


def test_cold_and_warm():
    """What lies in the L2 when a run starts changes the order of its copies, not its results."""
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for i in range(len(BATCHES)):
        s, c = batch(i)
        want = attend(c)
        for _ in range(30):
            flush.fill_(1)
            assert same(want, attend(c))
