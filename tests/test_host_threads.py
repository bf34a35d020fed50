"""Calls from several host threads at once.  The limit on a kernel's shared memory
is state of the process: what one call sets there must not fail the launch of
another call of another size."""
import threading

import pytest
import torch

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


def together(*works, calls=4000):
    """Each work on a thread and a stream of its own, `calls` times; the first error is raised."""
    errors, ready = [], threading.Barrier(len(works))
    torch.cuda.synchronize()

    def loop(work):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                ready.wait()
                for i in range(calls):
                    if errors:
                        return
                    work(i)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("rows,small,large", [(2, 1000, 128000), (2, 1000, 40000), (400, 900, 14000)])
@pytest.mark.parametrize("temperature", [0.0, 1.0])  # greedy: the GPU is not what the threads wait for
def test_vocabularies_of_two_sizes(rows, small, large, temperature):
    """Rows with an SM for each of their CTAs, and more rows than SMs."""
    g = torch.Generator(device="cuda").manual_seed(rows)

    def work_of(vocab):
        x = torch.randn((rows, vocab), generator=g, device="cuda")
        u = torch.rand((rows,), generator=g, device="cuda")
        want = ta.sample(x, u, temperature)
        got = [None]

        def work(i):
            got[0] = ta.sample(x, u, temperature)
            if i % 200 == 199:
                assert all(torch.equal(a, b) for a, b in zip(want, got[0]))
        return work

    together(work_of(small), work_of(large), work_of(small))
