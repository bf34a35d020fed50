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


def test_batches_of_two_sizes():
    def work_of(requests):
        lens = torch.arange(requests, device="cuda", dtype=torch.int32) % 32
        table = torch.arange(3 * requests, device="cuda", dtype=torch.int32).reshape(requests, 3)
        free = torch.arange(3 * requests, 4 * requests, device="cuda", dtype=torch.int32)
        n_free = torch.tensor([requests], device="cuda", dtype=torch.int32)
        new = torch.ones_like(lens)
        before = [x.clone() for x in (lens, free, n_free)]
        want = ta.extend_tables(lens, new, table, free, n_free, requests)
        ta.extend_tables(lens, -new, table, free, n_free, 0)

        def work(i):
            got = ta.extend_tables(lens, new, table, free, n_free, requests)
            ta.extend_tables(lens, back, table, free, n_free, 0)
            if i % 200 == 199:
                assert all(torch.equal(a, b) for a, b in zip((*want, *before), (*got, lens, free, n_free)))
        back = -new
        return work

    together(work_of(4000), work_of(16384), calls=2000)
