"""Log probabilities, entropy and top tokens against their definition in float64.

Tolerances, with U = 2^-24.  y = (x - max) / T in 32 bits: two or three roundings
of |y| (difference, 1 / T, product), 3 U |y|; as an argument of exp2 one more of
|y| log2 e, and exp2 itself 2^-22: a weight is off by e(y) = 4.5 U |y| + 2^-22 of
itself.  Weights matter up to |y| = 25 + ln(vocab) or so, and their sum's error is
the weighted mean of e(y), at most 2^-22 + 4.5 U * mean|y|, where the mean of |y|
under the weights is below the entropy; the sum of n terms in pieces of at most
1024 and a tree adds less than 1100 U only if all errors go one way: 2^-20 is
taken (round-off of either sign).  ln S: the same, and 2^-22 |ln S|.  So a log
probability is off by E = 3 U |y| + 2^-20 + 2^-22 (1 + ln S + H).  The entropy
ln S + D / S: D's terms w |y| are off by e(y) + 3 U each: by 2 E (1 + H)."""
import math

import numpy as np
import pytest
import torch

from oracle import drafts as oracle

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def check(x, given, temperature, top, got):
    """x [rows, vocab] on the CPU; temperature: one number or one a row."""
    rows, vocab = x.shape
    heat = [float(np.float32(t)) for t in (temperature if np.ndim(temperature) else [temperature] * rows)]
    lp, entropy, at, best = (None if g is None else g.cpu().double().numpy() for g in got)
    for r in range(rows):
        row = x[r].double().numpy()
        want, h, tops = oracle.token_logprobs(row, given[r], heat[r], top)
        if math.isnan(h):
            assert np.isnan(lp[r]).all() and math.isnan(entropy[r]) and np.isnan(best[r]).all() and (at[r] == -1).all()
            continue
        largest = max((b for _, b in tops[:1]), default=0.0)
        log_s = -largest if top else math.log(vocab)

        def bound(p):
            return 3 * 2.0 ** -24 * abs(p) + 2.0 ** -20 + 2.0 ** -22 * (1 + log_s + h)

        single = lambda p: float(np.float32(p))  # noqa: E731  (what lies past 32 bits is infinite there)
        for p, q in zip(map(single, want), lp[r]):
            assert (math.isnan(p) and math.isnan(q)) or p == q or abs(p - q) <= bound(p), (r, p, q)
        assert abs(entropy[r] - h) <= 2 * bound(0) * (1 + h), (r, entropy[r], h)
        assert at[r].tolist() == [i for i, _ in tops]
        for p, q in zip((single(b) for _, b in tops), best[r]):
            assert p == q or abs(p - q) <= bound(p), (r, p, q)


def run(x, given, temperature, top):
    heat = torch.tensor(temperature, dtype=torch.float32, device="cuda") if np.ndim(temperature) else temperature
    return ta.token_logprobs(x.cuda(), torch.tensor(given, dtype=torch.int32, device="cuda"), heat, top)


def logits(seed, rows, vocab, dtype, stride=None):
    g = torch.Generator().manual_seed(seed)
    x = 2.2 * torch.randn((rows, stride or vocab), generator=g)
    x[:, :: max(1, vocab // 11)] += 7
    return x.to(TYPES[dtype])[:, :vocab]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,stride,top", [
    (1, 1, None, 1), (1, 7, None, 3), (3, 33, 40, 5), (2, 1000, 1001, 64), (5, 4097, None, 1), (1, 32000, None, 20),
    (2, 50257, 50304, 8), (1, 262144, None, 64), (3, 262143, 262145, 5), (200, 700, 701, 16), (2, 17, None, 64), (9, 8191, 8192, 0)])
def test_against_the_definition(rows, vocab, stride, top, dtype):
    x = logits(rows + vocab, rows, vocab, dtype, stride)
    g = np.random.default_rng(vocab)
    given = g.integers(-1, vocab + 1, (rows, 3)).tolist()
    check(x, given, 1.0, top, run(x, given, 1.0, top))
    heat = (0.4 + g.random(rows)).tolist()
    check(x, given, heat, top, run(x, given, heat, top))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 40, 160, 700, 2000])
def test_many_rows(rows):
    x = logits(rows, rows, 2053, "bf16")
    given = np.random.default_rng(rows).integers(0, 2053, (rows, 1)).tolist()
    check(x, given, 0.7, 8, run(x, given, 0.7, 8))


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [40, 3001, 150000])
def test_masked_and_broken_rows(vocab):
    inf, nan = math.inf, math.nan
    x = logits(vocab, 12, vocab, "fp32")
    x[0, 1:] = -inf              # one token left
    x[1] = -inf                  # none
    x[2, vocab // 2] = nan
    x[3, vocab - 1] = inf        # all of the probability
    x[4, [1, vocab // 3]] = inf  # shared by two
    x[5] = 0.25                  # all equal: by index
    x[6, : vocab - 3] = -inf     # fewer than asked for
    x[7] = torch.finfo(torch.float32).min  # a mask's lowest value everywhere
    x[8, 2:] = torch.finfo(torch.float32).min
    x[9] = torch.linspace(-60, 60, vocab)          # ever larger: the list of the best changes all the time
    x[10] = torch.linspace(60, -60, vocab)
    x[11, ::2], x[11, 1::2] = -0.0, 0.0            # equal
    given = [[0, vocab - 1, vocab // 3]] * 12
    for top in (0, 5, 64):
        check(x, given, 1.0, top, run(x, given, 1.0, top))
    check(x, given, [0.3] * 12, 6, run(x, given, [0.3] * 12, 6))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_no_temperature_is_the_largest(dtype):
    x = logits(3, 4, 999, dtype)
    x[2, 300:] = x[2].max()
    given = [[int(x[r].argmax()), 5, 998] for r in range(4)]
    for heat in (0.0, -1.0, [0.0, 1.0, -2.0, math.nan]):
        check(x, given, heat, 4, run(x, given, heat, 4))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("heat", [1e-3, 1e4])
def test_sharp_and_flat(heat, dtype):
    x = logits(4, 3, 5000, dtype)
    given = [[1, 2, 3]] * 3
    check(x, given, heat, 5, run(x, given, heat, 5))


@pytest.mark.gpu
def test_ties_go_to_the_lowest_index():
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-3, 4, (6, 40000), generator=g).to(torch.bfloat16)
    given = [[0]] * 6
    check(x, given, 1.0, 64, run(x, given, 1.0, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("copies,top", [(1, 8), (1, 64), (300, 8), (300, 64)])
def test_rows_that_rise(copies, top, dtype):
    """The largest come last, in pieces of many sizes: what lies above the largest so far is few, many, all."""
    vocab = 40000
    i = torch.arange(vocab)
    noise = torch.randn((4, vocab), generator=torch.Generator().manual_seed(top))
    x = torch.stack([i * 1e-3, (i // 3000) * 1.5 + noise[0], torch.where(i % 2048 < 40, i * 2e-3, noise[1]),
                     torch.where((i > 9000) & (i < 17000), 8 + noise[2], noise[2]), torch.where(i > vocab - 1500, 9 + noise[3], noise[3])])
    x = x.to(TYPES[dtype])
    given = [[0, vocab - 1]] * len(x)
    got = run(x.repeat(copies, 1), given * copies, 1.3, top)
    check(x, given, 1.3, top, [g[:len(x)] for g in got])
    for g in got:  # (other rows at other alignments of the grid, the same sums)
        assert torch.equal(g.reshape(copies, -1), g[:len(x)].reshape(1, -1).expand(copies, -1))


@pytest.mark.gpu
def test_largest_values():
    big = torch.finfo(torch.float32).max
    x = torch.zeros((3, 5000))
    x[0, 7], x[0, 8] = big, -big
    x[1] = -big
    x[1, 4999] = big
    x[2] = big
    given = [[7, 8, 4999]] * 3
    check(x, given, 1.0, 3, run(x, given, 1.0, 3))


@pytest.mark.gpu
def test_forms_of_the_arguments():
    x = logits(9, 5, 600, "fp32").cuda()
    tokens = torch.arange(5, dtype=torch.int32, device="cuda")
    one = ta.token_logprobs(x, tokens)
    two = ta.token_logprobs(x, tokens[:, None], temperature=None, top=3)
    assert one[0].shape == (5,) and torch.equal(one[0], two[0][:, 0]) and torch.equal(one[1], two[1])
    assert one[2].shape == (5, 0) and one[3].shape == (5, 0)
    none = ta.token_logprobs(x, top=3)
    assert none[0] is None and torch.equal(none[2], two[2]) and torch.equal(none[3], two[3])
    empty = ta.token_logprobs(x[:0], tokens[:0], top=2)
    assert [tuple(e.shape) for e in empty] == [(0,), (0,), (0, 2), (0, 2)]
    assert ta.token_logprobs(x, tokens.reshape(5, 1)[:, :0])[0].shape == (5, 0)
    # a row alone gives what it gives among others
    for r in range(5):
        alone = ta.token_logprobs(x[r:r + 1], tokens[r:r + 1], top=3)
        assert torch.equal(alone[2], two[2][r:r + 1])


@pytest.mark.gpu
def test_streams_graphs_and_same_results_again():
    x = logits(11, 30, 9000, "bf16").cuda()
    tokens = torch.arange(30, dtype=torch.int32, device="cuda")
    first = ta.token_logprobs(x, tokens, 0.9, 9)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = [ta.token_logprobs(x, tokens, 0.9, 9, stream=s) for s in (stream, None, stream.cuda_stream)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        runs.append(ta.token_logprobs(x, tokens, 0.9, 9))
    graph.replay()
    torch.cuda.synchronize()
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    x.copy_(logits(12, 30, 9000, "bf16").cuda())
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(runs[-1], ta.token_logprobs(x, tokens, 0.9, 9)))


# ------------------------------------------------------------- refusals (no GPU)
def _run(**kw):
    a = dict(logits=256, stride=100, dtype=0, rows=2, vocab=100, given=256, n_given=1, heat=None, heat_all=1.0, top=3, lp=256,
             entropy=256, at=256, best=256, stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_token_logprobs(*a.values())


@pytest.mark.parametrize("kw,name", [
    (dict(logits=None), "INVALID_ARG"), (dict(given=None), "INVALID_ARG"), (dict(lp=None), "INVALID_ARG"),
    (dict(at=None), "INVALID_ARG"), (dict(best=None), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"),
    (dict(vocab=0), "INVALID_ARG"), (dict(n_given=-1), "INVALID_ARG"), (dict(top=-1), "INVALID_ARG"),
    (dict(stride=99), "INVALID_ARG"), (dict(dtype=3), "UNSUPPORTED"), (dict(vocab=262145, stride=262145), "UNSUPPORTED"),
    (dict(top=65), "UNSUPPORTED"), (dict(rows=1 << 28), "UNSUPPORTED"), (dict(logits=257), "ALIGNMENT"),
    (dict(logits=258, dtype=2), "ALIGNMENT"), (dict(heat=2), "ALIGNMENT"), (dict(best=258), "ALIGNMENT")])
def test_refusals(kw, name):
    assert _abi.STATUS_NAMES[_run(**kw)] == "TA_ERR_" + name
    assert _abi.load_library().tree_attn_last_error()


def test_host_tensors_and_large_numbers_are_refused():
    x = torch.zeros((2, 5))
    with pytest.raises(ValueError, match="CUDA"):
        ta.token_logprobs(x)
    for top in (2 ** 31, -1):
        with pytest.raises(ValueError, match="top"):
            ta.token_logprobs(x, top=top)
    with pytest.raises(ValueError, match="32 bits"):
        ta.token_logprobs(torch.empty((2 ** 32 + 1, 1), device="meta"))


@pytest.mark.gpu
def test_wrong_tensors_are_refused():
    x, z = torch.zeros((2, 6), device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for args in ((x.double(), z), (x[0], z), (x[:, ::2], z), (x, z[:1]), (x, z.long()), (x, z.cpu()), (x, z, z), (x, z, x[0])):
        with pytest.raises(ValueError):
            ta.token_logprobs(*args)
    with pytest.raises(ta.TreeAttnError):
        ta.token_logprobs(x, z, top=65)
