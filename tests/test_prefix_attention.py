"""Attention of a batch behind a shared prefix, against its definition in
float64 on the same inputs.

Tolerances.  Let eps be half a step of the type (bf16 2^-8, fp16 2^-11).  The
output is rounded once (eps |out|), each weight once before the product with V
(eps times the mean A of |v| under the weights, plus, in fp16, half its
smallest step 2^-25 per key where a weight is subnormal).  A score is a sum of
d products in 32 bits: off by at most (d + 4) 2^-24 times scale * sum |q k|, X
below, which enters a weight relatively and so the output as 2 X A, and lse as
X.  exp2 is off by 2^-22 relatively, and its argument (up to |s| log2 e) by
2^-23 of itself; sums of n weights by less than 2^-20 with the pairing used."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import batch as oracle

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8, 0.0), "fp16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}


def make(seed, lens, new, hq, hkv, d, prefix, dtype="bf16", padding=0, width=None, tail=float("nan"), gain=1.0):
    """A batch with shuffled pages; slots past an end hold `tail`.  new: queries of each request (None: one each, no cu)."""
    kind = TYPES[dtype][0]
    g = torch.Generator().manual_seed(seed)
    pages = lambda n: -(-n // 16)  # noqa: E731
    width = max([1] + [pages(n) for n in lens]) if width is None else width
    total = pages(prefix) + sum(pages(n) for n in lens) + 2
    order = torch.randperm(total, generator=g).tolist()
    k = (gain * torch.randn((total, hkv, 16, d), generator=g)).to(kind)
    v = torch.randn((total, hkv, 16, d), generator=g).to(kind)
    take = lambda n: [order.pop() for _ in range(pages(n))]  # noqa: E731

    def end(ids, n):
        if n % 16:
            k[ids[-1], :, n % 16:], v[ids[-1], :, n % 16:] = tail, tail
        return ids

    pre = end(take(prefix), prefix)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        ids = end(take(n), n)
        table[b, : len(ids)] = torch.tensor(ids, dtype=torch.int32)
    cu = np.concatenate([[0], np.cumsum([1] * len(lens) if new is None else new)]).astype(int)
    tokens = int(cu[-1]) + padding
    q = torch.randn((tokens, hq + 3, d), generator=g).to(kind)[:, 1:hq + 1]
    ints = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return dict(q=q, k=k, v=v, table=table, lens=ints(lens), cu=None if new is None else ints(cu), pre=ints(pre),
                prefix=prefix, cu_all=cu, dtype=dtype)


def to_gpu(s):
    return {n: x.cuda() if torch.is_tensor(x) else x for n, x in s.items()}


def attend(c, **kw):
    return ta.prefix_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["cu"], c["pre"], c["prefix"], **kw)


def check(s, out, lse, scale=None):
    _, eps, tiny = TYPES[s["dtype"]]
    q, k = s["q"].double().numpy(), s["k"].double().nan_to_num(0).numpy()
    v = s["v"].double().nan_to_num(0).numpy()
    d = q.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    args = (s["table"].numpy(), s["lens"].numpy(), s["cu_all"], s["pre"].numpy(), s["prefix"], scale)
    want, want_lse = oracle.prefix_attention(q, k, v, *args)
    mean, _ = oracle.prefix_attention(q, k, np.abs(v), *args)
    x = (d + 4) * 2.0 ** -24 * scale * np.abs(q).sum(2).max(initial=0) * np.abs(k).max(initial=0)
    seen = np.isfinite(want_lse)
    big = np.abs(want_lse[seen]).max(initial=1) * 3
    x += big * 2.0 ** -22 + 2.0 ** -20
    n = s["prefix"] + int(s["lens"].max()) if len(s["lens"]) else 0
    tol = 1.02 * eps * (np.abs(want) + mean) + 2 * x * mean + n * tiny * np.abs(v).max(initial=0)
    err = np.abs(out.double().cpu().numpy() - want)
    assert not np.isnan(err).any()
    assert (err <= tol).all(), float((err - tol).max())
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), ~seen)
    assert np.abs(got[seen] - want_lse[seen]).max(initial=0) <= x


CASES = [
    # lens, queries (None: one each), heads, kv heads, d, prefix
    ([1], None, 1, 1, 64, 0),
    ([1], None, 4, 4, 64, 1),
    ([5, 16, 17, 1], None, 4, 4, 64, 256),
    ([5, 16, 17, 1], None, 8, 2, 128, 15),
    ([31, 0, 48, 33, 7], None, 32, 8, 128, 16),       # one request holds nothing: it sees the prefix alone
    ([31, 0, 48, 33, 7], None, 5, 5, 128, 0),         # ... or nothing at all
    ([700, 3, 90], [4, 1, 2], 64, 4, 128, 131),       # 64 rows: several row tiles
    ([40, 25, 9, 64], [3, 0, 5, 1], 12, 2, 64, 77),   # a request that sits the step out, 6 heads a kv head
    ([20, 90], [20, 17], 16, 1, 128, 40),             # a whole prompt at once, behind the prefix
    ([3], [5], 8, 8, 64, 4),                          # more queries than tokens: the first see the prefix alone
    ([130, 2, 65], [1, 2, 1], 128, 1, 64, 300),       # 128 heads a kv head
    ([200, 1], None, 28, 4, 128, 1000),               # 7 heads a kv head
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_definition(case, dtype):
    lens, new, hq, hkv, d, prefix = CASES[case]
    s = make(case, lens, new, hq, hkv, d, prefix, dtype, padding=0 if new is None else 3, width=60)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(to_gpu(s), status=status)
    assert out.dtype == s["q"].dtype and status.item() == 0
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,prefix,heads", [([6000] + [1] * 30, 0, (8, 2)), ([3000, 2999, 5], 17, (4, 4)),
                                               ([37] * 300, 64, (8, 2)), (list(range(1, 130)), 5000, (4, 1)),
                                               ([1], 20000, (2, 1))])
def test_work_cut_into_runs(lens, prefix, heads):
    """Long and short requests together, long prefixes: segments in one run, in two, and in hundreds."""
    s = make(len(lens), lens, None, *heads, 128, prefix)
    out, lse = attend(to_gpu(s))
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,heads,prefix", [
    ([100] * 40, None, (16, 4), 40001),                  # tiles beside the own pages, and behind them
    ([700] * 9, None, (32, 8), 12000),
    ([30] * 64, [3] * 64, (16, 2), 10000),               # own tiles of 16 rows
    ([2000] * 60, [2] * 60, (24, 4), 500),               # own pages first, on all SMs
    ([3000] * 40, None, (4, 2), 140),
    ([0] * 50, None, (8, 2), 3000)])                     # no own pages at all
def test_sms_shared_by_tiles_and_own_pages(lens, new, heads, prefix):
    s = make(prefix, lens, new, *heads, 128, prefix)
    out, lse = attend(to_gpu(s))
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [383, 384, 385, 2500])
@pytest.mark.parametrize("asking,heads,prefix", [(1, (16, 1), 700), (5, (4, 2), 33), (9, (2, 2), 9000), (300, (4, 2), 50)])
def test_a_few_of_many_requests_ask(requests, asking, heads, prefix):
    """Up to 16 query rows behind a prefix stand in one line with the requests' own pages; more go apart."""
    new = [0] * requests
    for i in range(asking):
        new[(i + 1) * requests // asking - 1] = 1
    s = make(requests, [(7 * b) % 40 for b in range(requests)], new, *heads, 128, prefix, padding=2)
    out, lse = attend(to_gpu(s))
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("requests,prefix", [(2049, 20), (5000, 0), (3000, 150)])
def test_more_requests_than_a_cta_searches_by_itself(requests, prefix):
    g = np.random.default_rng(requests)
    lens, new = g.integers(0, 40, requests).tolist(), g.integers(0, 2, requests).tolist()
    s = make(requests, lens, new, 2, 1, 64, prefix, padding=5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(to_gpu(s), status=status)
    assert status.item() == 0
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 33, 900])
def test_captured_and_replayed_with_other_lengths(prefix):
    """A graph's runs follow the lengths, offsets and tables that lie in memory when it is replayed."""
    s = make(9, [100, 7, 60], [2, 1, 1], 12, 2, 64, prefix, padding=2, width=9)
    c = to_gpu(s)
    attend(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attend(c)
    for lens, cu in (([100, 7, 60], [0, 2, 3, 4]), ([90, 0, 48], [0, 1, 1, 6]), ([1, 2, 3], [0, 0, 3, 6]), ([0, 0, 0], [0, 0, 0, 0])):
        out.fill_(7)
        lse.fill_(7)
        for name, x in (("lens", lens), ("cu", cu)):
            s[name] = torch.tensor(x, dtype=torch.int32)
            c[name].copy_(s[name])
        s["cu_all"] = np.array(cu)
        graph.replay()
        check(s, out, lse)


@pytest.mark.gpu
def test_scale_and_large_scores():
    s = make(3, [100, 64], None, 4, 2, 64, 90, gain=3.0)
    out, lse = attend(to_gpu(s), softmax_scale=0.31)
    check(s, out, lse, scale=0.31)


@pytest.mark.gpu
def test_given_outputs_no_lse_and_a_table_view():
    s = make(4, [33, 80, 5], [2, 1, 1], 8, 2, 128, 30, padding=2)
    c = to_gpu(s)
    wide = torch.full((3, 30), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + c["table"].shape[1]] = c["table"]
    c["table"] = wide[:, 3:20]
    out, lse = torch.full((6, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((6, 8), 7.0, device="cuda")
    got = attend(c, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check(s, out, lse)
    assert (out[4:] == 0).all() and torch.isneginf(lse[4:]).all()  # tokens of no request
    again, none = attend(c, want_lse=False)
    assert none is None and torch.equal(again, out)


@pytest.mark.gpu
def test_masked_values_do_not_count():
    """Infinities in K where a draft does not look yet, the largest finite values in V there."""
    s = make(5, [40], [4], 4, 2, 64, 20)
    s["k"][s["table"][0, 2], :, 6:8] = float("inf")     # the last two drafts' keys
    s["v"][s["table"][0, 2], :, 6:8] = torch.finfo(torch.bfloat16).max
    c = to_gpu(s)
    out, lse = attend(c)
    s["cu_all"] = np.array([0, 2])
    s["lens"] = torch.tensor([38], dtype=torch.int32)
    s["k"] = torch.where(s["k"].isinf(), 0, s["k"])
    s["q"] = s["q"][:2]
    check(s, out[:2], lse[:2])


@pytest.mark.gpu
def test_bad_values_on_the_device_are_said_and_stay_in_bounds():
    s = make(6, [40, 50], None, 4, 2, 64, 33)
    for name, at, value, bit in (("table", (0, 1), 10 ** 6, _abi.BATCH_BAD_SLOT), ("table", (1, 0), -5, _abi.BATCH_BAD_SLOT),
                                 ("pre", (2,), 99, _abi.BATCH_BAD_SLOT), ("lens", (0,), -3, _abi.BATCH_BAD_INPUT),
                                 ("lens", (1,), 10 ** 6, _abi.BATCH_BAD_INPUT)):
        c = to_gpu(s)
        c[name] = c[name].clone()
        c[name][at] = value
        if name == "lens" and value > 0:
            c["table"] = torch.zeros_like(c["table"])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        attend(c, status=status)
        assert status.item() == bit
    for cu in ([0, 5, 2], [-1, 1, 2], [0, 1, 3], [2, 1, 0], [0, 2, 1], [0, 2, -9]):
        c = to_gpu(s)
        c["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        attend(c, status=status)
        assert status.item() == _abi.BATCH_BAD_INPUT
    # a page out of range reads as zeros
    c = to_gpu(s)
    c["table"][0, 1] = 10 ** 6
    out, lse = attend(c)
    s["table"][0, 1] = len(s["k"])
    s["k"], s["v"] = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (s["k"], s["v"]))
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [40, 600])
@pytest.mark.parametrize("prefix", [0, 5, 500])
def test_offsets_out_of_order_give_no_token_a_request(requests, prefix):
    """Offsets that give all tokens to every second request, over and over: no such work is done."""
    s = make(requests, [90] * requests, [1] * 4 + [0] * (requests - 4), 16 if prefix == 500 else 4, 2, 64, prefix)
    c = to_gpu(s)
    c["cu"] = torch.tensor(([0, 4] * requests)[: requests + 1], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(c, status=status)
    assert status.item() == _abi.BATCH_BAD_INPUT
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.gpu
def test_no_request_no_token():
    s = to_gpu(make(7, [4], None, 4, 2, 64, 10))
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, lse = ta.prefix_attention(s["q"][:0], s["k"], s["v"], s["table"][:0], z, None, s["pre"], 10)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = ta.prefix_attention(s["q"], s["k"], s["v"], s["table"][:0], z, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                   s["pre"], 10)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.gpu
def test_streams_and_same_results_again():
    s = make(8, [300, 20, 1000], None, 8, 2, 128, 700)
    c = to_gpu(s)
    a = attend(c)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = [attend(c, stream=st) for st in (stream, None, stream.cuda_stream, None)]  # two streams at once
    torch.cuda.synchronize()
    for out, lse in runs:
        assert torch.equal(out, a[0]) and torch.equal(lse, a[1])
    check(s, *a)


# ------------------------------------------------------------- refusals (no GPU)
def _run(**kw):
    a = dict(q=256, q_stride=512, k=256, v=256, pages=4, table=256, stride=4, width=4, lens=256, cu=256, b=2, t=2, pre=256,
             prefix=10, hq=4, hkv=2, d=128, dtype=0, scale=0.0, out=256, lse=256, status=None, work=256, bytes=1 << 40,
             stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_prefix_run(*a.values())


@pytest.mark.parametrize("kw,name", [
    (dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(lens=None), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"), (dict(pre=None), "INVALID_ARG"),
    (dict(work=None), "INVALID_ARG"), (dict(b=-1), "INVALID_ARG"), (dict(t=-1), "INVALID_ARG"),
    (dict(prefix=-1), "INVALID_ARG"), (dict(hkv=0), "INVALID_ARG"), (dict(pages=0), "INVALID_ARG"),
    (dict(stride=3), "INVALID_ARG"), (dict(q_stride=504), "INVALID_ARG"), (dict(cu=None, t=3), "INVALID_ARG"),
    (dict(width=-1), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"), (dict(hq=5), "UNSUPPORTED"),
    (dict(hq=258), "UNSUPPORTED"), (dict(dtype=2), "UNSUPPORTED"), (dict(b=16385), "UNSUPPORTED"),
    (dict(pages=-1), "UNSUPPORTED"), (dict(width=1 << 27, stride=1 << 27), "UNSUPPORTED"),
    (dict(t=1 << 29), "UNSUPPORTED"), (dict(t=1 << 24, b=9, width=1 << 26, stride=1 << 26), "UNSUPPORTED"), (dict(q=264), "ALIGNMENT"), (dict(q_stride=516), "ALIGNMENT"),
    (dict(lens=258), "ALIGNMENT"), (dict(work=272), "ALIGNMENT"), (dict(bytes=100), "BUFFER_TOO_SMALL")])
def test_refusals(kw, name):
    assert _abi.STATUS_NAMES[_run(**kw)] == "TA_ERR_" + name
    assert _abi.load_library().tree_attn_last_error()


def test_workspace_grows_with_the_batch():
    f, n = _abi.load_library().tree_attn_prefix_workspace, ctypes.c_size_t(0)
    sizes = []
    for t in (0, 1, 100):
        assert f(t, t, 50, 8, 2, 128, ctypes.byref(n)) == _abi.TA_OK
        sizes.append(n.value)
    assert sizes[0] == 0 and sizes[1] < sizes[2]
    assert _abi.STATUS_NAMES[f(1, 1, 1, 3, 2, 128, ctypes.byref(n))] == "TA_ERR_UNSUPPORTED"
    assert _abi.STATUS_NAMES[f(1, 1, 1, 2, 2, 128, None)] == "TA_ERR_INVALID_ARG"


def test_host_tensors_are_refused():
    s = make(1, [4], None, 4, 2, 64, 10)
    with pytest.raises(ValueError, match="CUDA"):
        attend(s)


@pytest.mark.gpu
def test_wrong_tensors_are_refused():
    s = to_gpu(make(2, [4, 9], None, 4, 2, 64, 10))
    for change in (dict(q=s["q"].half()), dict(q=s["q"].transpose(0, 1)), dict(q=s["q"][..., :32]), dict(v=s["v"][:-1]),
                   dict(table=s["table"][:1]), dict(lens=s["lens"].long()), dict(prefix=200), dict(pre=None),
                   dict(cu=s["lens"])):
        with pytest.raises(ValueError):
            attend({**s, **change})
    with pytest.raises(ValueError):
        attend(s, out=torch.empty(2, 4, 64, device="cuda"))
    with pytest.raises(ta.TreeAttnError):
        attend({**s, "q": s["q"][:1]})
