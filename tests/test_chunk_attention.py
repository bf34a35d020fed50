"""Attention of prompts and of trees of drafted tokens over their pages, against
the definition in float64 on the same inputs.

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

from oracle import drafts as oracle

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8, 0.0), "fp16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}


def tree(seed, n, kind="mixed"):
    """Parents of n nodes."""
    g = np.random.default_rng(seed)
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return ([-1] + [0] * n)[:n]
    if kind == "roots":
        return [-1] * n
    return [-1 if i == 0 or g.random() < 0.05 else i - 1 if g.random() < 0.3 else int(g.integers(0, i)) for i in range(n)]


def make(seed, lens, new, hq, hkv, d, dtype="bf16", trees=None, padding=0, width=None, tail=float("nan"), gain=1.0):
    """A batch with shuffled pages; slots past an end hold `tail`.  new: new tokens of each request (None: one each, no cu);
    trees: None (causal), or the kind of each request's tree."""
    kind = TYPES[dtype][0]
    g = torch.Generator().manual_seed(seed)
    pages = lambda n: -(-max(n, 0) // 16)  # noqa: E731
    width = max([1] + [pages(n) for n in lens]) if width is None else width
    total = sum(pages(n) for n in lens) + 2
    order = torch.randperm(total, generator=g).tolist()
    k = (gain * torch.randn((total, hkv, 16, d), generator=g)).to(kind)
    v = torch.randn((total, hkv, 16, d), generator=g).to(kind)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        ids = [order.pop() for _ in range(pages(n))]
        if n % 16:
            k[ids[-1], :, n % 16:], v[ids[-1], :, n % 16:] = tail, tail
        table[b, : len(ids)] = torch.tensor(ids, dtype=torch.int32)
    counts = [1] * len(lens) if new is None else new
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    tokens = int(cu[-1]) + padding
    q = torch.randn((tokens, hq + 3, d), generator=g).to(kind)[:, 1:hq + 1]
    ints = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    parents = None
    if trees is not None:
        parents = ints(sum((tree(seed + b, n, trees) for b, n in enumerate(counts)), []) + [-7] * padding)
    return dict(q=q, k=k, v=v, table=table, lens=ints(lens), cu=None if new is None else ints(cu), parents=parents, cu_all=cu,
                dtype=dtype)


def to_gpu(s):
    return {n: x.cuda() if torch.is_tensor(x) else x for n, x in s.items()}


def attend(c, **kw):
    args = c["q"], c["k"], c["v"], c["table"], c["lens"]
    if c["parents"] is None:
        return ta.prompt_attention(*args, c["cu"], **kw)
    return ta.draft_attention(*args, c["parents"], c["cu"], **kw)


def check(s, out, lse, scale=None):
    _, eps, tiny = TYPES[s["dtype"]]
    q, k = s["q"].double().numpy(), s["k"].double().nan_to_num(0).numpy()
    v = s["v"].double().nan_to_num(0).numpy()
    d = q.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    parents = None if s["parents"] is None else s["parents"].tolist()
    args = (s["table"].numpy(), s["lens"].numpy(), s["cu_all"], parents, scale)
    want, want_lse = oracle.chunk_attention(q, k, v, *args)
    mean, _ = oracle.chunk_attention(q, k, np.abs(v), *args)
    x = (d + 4) * 2.0 ** -24 * scale * np.abs(q).sum(2).max(initial=0) * np.abs(k).max(initial=0)
    seen = np.isfinite(want_lse)
    big = np.abs(want_lse[seen]).max(initial=1) * 3
    x += big * 2.0 ** -22 + 2.0 ** -20
    n = int(s["lens"].max()) if len(s["lens"]) else 0
    tol = 1.02 * eps * (np.abs(want) + mean) + 2 * x * mean + n * tiny * np.abs(v).max(initial=0)
    err = np.abs(out.double().cpu().numpy() - want)
    assert not np.isnan(err).any()
    assert (err <= tol).all(), float((err - tol).max())
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), ~seen)
    assert np.abs(got[seen] - want_lse[seen]).max(initial=0) <= x


CASES = [
    # lens, new tokens (None: one each), heads, kv heads, d
    ([1], None, 1, 1, 64),
    ([1], [1], 4, 4, 128),
    ([5, 16, 17, 1], None, 8, 2, 128),
    ([31, 0, 48, 33, 7], [2, 0, 48, 1, 7], 32, 8, 128),     # one request holds nothing, two are whole prompts
    ([700, 3, 90], [4, 1, 2], 64, 4, 128),
    ([40, 25, 9, 64], [3, 0, 5, 1], 12, 2, 64),             # a request that sits the step out, 6 heads a kv head
    ([75, 127, 128, 129], [75, 127, 128, 129], 8, 4, 64),   # prompts that end around a step's end
    ([3], [5], 8, 8, 64),                                   # more new tokens than tokens: the first see nothing
    ([2, 300], [120, 1], 4, 2, 64),                         # ... nearly all of them
    ([0, 40], [3, 40], 4, 4, 128),                          # nothing held, and queries
    ([130, 2, 65], [1, 2, 1], 128, 1, 64),                  # 128 heads a kv head
    ([200, 90], [100, 90], 28, 4, 128),                     # 7 heads a kv head: blocks of 36 tokens
    ([400, 9], [128, 9], 10, 2, 64),                        # 5 heads
    ([900], [127], 3, 1, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("trees", [None, "mixed"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_definition(case, trees, dtype):
    lens, new, hq, hkv, d = CASES[case]
    if trees is not None and new is not None:
        lens = [n - max(0, m - 128) for n, m in zip(lens, new)]
        new = [min(m, 128) for m in new]
    s = make(case, lens, new, hq, hkv, d, dtype, trees, padding=0 if new is None else 3, width=60)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(to_gpu(s), status=status)
    assert out.dtype == s["q"].dtype and status.item() == 0
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,heads,d", [
    ([6000] + [1] * 30, [1] * 31, (8, 2), 128),             # one long request: cut into many pieces
    ([1500, 1000], [1500, 700], (8, 2), 64),
    ([1300], [1300], (5, 1), 128),
    ([37] * 300, [3] * 300, (8, 2), 64),
    (list(range(1, 130)), list(range(1, 130)), (4, 1), 64),
    ([20000], [2], (2, 1), 128),
    ([9000, 4100], [30, 100], (16, 2), 128),
    ([2048] * 3, [64] * 3, (32, 1), 64),                    # 2048 rows a kv head
])
def test_work_cut_into_runs(lens, new, heads, d):
    """Long and short requests together: segments in one run, in two, and in hundreds."""
    for trees in (None, "mixed") if max(new) <= 128 else (None,):
        s = make(len(lens), lens, new, *heads, d, trees=trees, padding=1)
        out, lse = attend(to_gpu(s))
        check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["chain", "star", "roots", "mixed"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 96, 128])
def test_shapes_of_trees(kind, n):
    """Trees whose nodes cross words of the mask, pages and steps: the first node sits at all places of a page."""
    s = make(n, [n + held for held in (0, 1, 15, 16, 113, 127, 130)], [n] * 7, 4, 2, 64, trees=kind)
    out, lse = attend(to_gpu(s))
    check(s, out, lse)
    if kind == "chain":  # what a causal chunk sees
        out2, lse2 = attend(to_gpu({**s, "parents": None}))
        check({**s, "parents": None}, out, lse)
        check({**s, "parents": None}, out2, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [1, 383, 384, 385, 5000])
def test_many_requests(requests):
    g = np.random.default_rng(requests)
    new = g.integers(0, 3, requests).tolist()
    lens = [int(m + g.integers(0, 40)) for m in new]
    s = make(requests, lens, new, 2, 1, 64, trees="mixed", padding=5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(to_gpu(s), status=status)
    assert status.item() == 0
    check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("trees", [None, "mixed"])
def test_captured_and_replayed_with_other_lengths(trees):
    """A graph's runs follow the lengths, offsets, trees and tables that lie in memory when it is replayed."""
    s = make(9, [100, 70, 160], [20, 41, 60], 12, 2, 64, trees=trees, padding=2, width=12)
    c = to_gpu(s)
    attend(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attend(c)
    for lens, cu in (([100, 70, 160], [0, 20, 61, 121]), ([90, 0, 160], [0, 1, 1, 123]), ([1, 2, 3], [0, 0, 3, 6]), ([0, 0, 0], [0, 0, 0, 0])):
        out.fill_(7)
        lse.fill_(7)
        for name, x in (("lens", lens), ("cu", cu)):
            s[name] = torch.tensor(x, dtype=torch.int32)
            c[name].copy_(s[name])
        if trees:
            p = sum((tree(b, cu[b + 1] - cu[b]) for b in range(3)), [])
            s["parents"] = torch.tensor(p + [-1] * (len(c["q"]) - len(p)), dtype=torch.int32)
            c["parents"].copy_(s["parents"])
        s["cu_all"] = np.array(cu)
        graph.replay()
        check(s, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("trees", [None, "mixed"])
def test_scale_and_large_scores(trees):
    s = make(3, [100, 64], [30, 64], 4, 2, 64, gain=3.0, trees=trees)
    out, lse = attend(to_gpu(s), softmax_scale=0.31)
    check(s, out, lse, scale=0.31)


@pytest.mark.gpu
def test_a_growing_maximum():
    """Keys whose scores rise along the sequence: the accumulators are rescaled in every step."""
    s = make(12, [900], [40], 4, 1, 128)
    q = torch.ones_like(s["q"])
    s["q"] = q
    for j in range(900):
        s["k"][s["table"][0, j // 16], :, j % 16] = j / 20
    out, lse = attend(to_gpu(s))
    check(s, out, lse)


@pytest.mark.gpu
def test_given_outputs_no_lse_and_a_table_view():
    s = make(4, [33, 80, 5], [20, 30, 1], 8, 2, 128, padding=2)
    c = to_gpu(s)
    wide = torch.full((3, 30), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + c["table"].shape[1]] = c["table"]
    c["table"] = wide[:, 3:20]
    out, lse = torch.full((53, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((53, 8), 7.0, device="cuda")
    got = attend(c, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check(s, out, lse)
    assert (out[51:] == 0).all() and torch.isneginf(lse[51:]).all()  # tokens of no request
    again, none = attend(c, want_lse=False)
    assert none is None and torch.equal(again, out)


@pytest.mark.gpu
@pytest.mark.parametrize("trees", [None, "star"])
def test_masked_values_do_not_count(trees):
    """Infinities in K where a query does not look, the largest finite values in V there."""
    s = make(5, [40], [4], 4, 2, 64, trees=trees)
    big = torch.finfo(torch.bfloat16).max
    s["k"][s["table"][0, 2], :, 7] = float("inf")       # the last new token's key
    s["v"][s["table"][0, 2], :, 7] = big
    out, lse = attend(to_gpu(s))
    s["k"][s["table"][0, 2], :, 7] = 0
    s["v"][s["table"][0, 2], :, 7] = 0
    s["cu_all"] = np.array([0, 4])
    s["q"], out, lse = s["q"][:3], out[:3], lse[:3]
    s["cu_all"] = np.array([0, 3])
    s["lens"] = torch.tensor([39], dtype=torch.int32)
    if trees:
        s["parents"] = s["parents"][:3]
    check(s, out, lse)


@pytest.mark.gpu
def test_bad_values_on_the_device_are_said_and_stay_in_bounds():
    for trees in (None, "mixed"):
        s = make(6, [40, 50], [4, 9], 4, 2, 64, trees=trees)
        for name, at, value, bit in (("table", (0, 1), 10 ** 6, _abi.BATCH_BAD_SLOT), ("table", (1, 0), -5, _abi.BATCH_BAD_SLOT),
                                     ("lens", (0,), -3, _abi.BATCH_BAD_INPUT), ("lens", (1,), 10 ** 6, _abi.BATCH_BAD_INPUT)):
            c = to_gpu(s)
            c[name] = c[name].clone()
            c[name][at] = value
            if name == "lens" and value > 0:
                c["table"] = torch.zeros_like(c["table"])
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            attend(c, status=status)
            assert status.item() == bit
        for cu in ([0, 5, 2], [-1, 1, 2], [0, 1, 14], [2, 1, 0], [0, 2, 1], [0, 2, -9]):
            c = to_gpu(s)
            c["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            out, lse = attend(c, status=status)
            assert status.item() == _abi.BATCH_BAD_INPUT
            assert not out.any() and torch.isneginf(lse).all()
        # a page out of range reads as zeros
        c = to_gpu(s)
        c["table"] = c["table"].clone()
        c["table"][0, 1] = 10 ** 6
        out, lse = attend(c)
        s["table"][0, 1] = len(s["k"])
        s["k"], s["v"] = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (s["k"], s["v"]))
        check(s, out, lse)


@pytest.mark.gpu
def test_parents_out_of_order_and_trees_too_large():
    s = make(7, [60, 300, 70], [20, 129, 9], 4, 2, 64)
    parents = tree(1, 20) + [-1] * 129 + tree(2, 9)
    parents[5], parents[9], parents[155] = 5, 4000, -9  # itself, far above, below -1: as if they had none
    c = to_gpu(s)
    c["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(c, status=status)
    assert status.item() == _abi.BATCH_BAD_INPUT
    assert not out[20:149].any() and torch.isneginf(lse[20:149]).all()  # a request of 129 nodes
    s["parents"] = torch.tensor(parents, dtype=torch.int32)
    keep = list(range(20)) + list(range(149, 158))
    s["q"], s["parents"], s["cu_all"] = s["q"][keep], s["parents"][keep], np.array([0, 20, 20, 29])
    check(s, out[keep], lse[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [40, 600])
def test_offsets_out_of_order_give_no_token_a_request(requests):
    """Offsets that give all tokens to every second request, over and over: no such work is done."""
    s = make(requests, [90] * requests, [1] * 4 + [0] * (requests - 4), 4, 2, 64)
    c = to_gpu(s)
    c["cu"] = torch.tensor(([0, 4] * requests)[: requests + 1], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = attend(c, status=status)
    assert status.item() == _abi.BATCH_BAD_INPUT
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.gpu
def test_no_request_no_token():
    s = to_gpu(make(7, [4], None, 4, 2, 64))
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    for f, more in ((ta.prompt_attention, ()), (ta.draft_attention, (z,))):
        out, lse = f(s["q"][:0], s["k"], s["v"], s["table"][:0], z, *more, None)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = ta.prompt_attention(s["q"], s["k"], s["v"], s["table"][:0], z, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.gpu
def test_streams_and_same_results_again():
    s = make(8, [300, 20, 1000], [80, 20, 70], 8, 2, 128, trees="mixed")
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
    a = dict(q=256, q_stride=512, k=256, v=256, pages=4, table=256, stride=4, width=4, lens=256, cu=256, parents=None, b=2, t=2,
             hq=4, hkv=2, d=128, dtype=0, scale=0.0, out=256, lse=256, status=None, work=256, bytes=1 << 40, stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_chunk_run(*a.values())


@pytest.mark.parametrize("kw,name", [
    (dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(lens=None), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"), (dict(b=-1), "INVALID_ARG"),
    (dict(t=-1), "INVALID_ARG"), (dict(hkv=0), "INVALID_ARG"), (dict(pages=0), "INVALID_ARG"),
    (dict(stride=3), "INVALID_ARG"), (dict(q_stride=504), "INVALID_ARG"), (dict(cu=None, t=3), "INVALID_ARG"),
    (dict(width=-1), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"), (dict(hq=5), "UNSUPPORTED"),
    (dict(hq=258), "UNSUPPORTED"), (dict(dtype=2), "UNSUPPORTED"), (dict(b=16385), "UNSUPPORTED"),
    (dict(pages=-1), "UNSUPPORTED"), (dict(width=1 << 27, stride=1 << 27), "UNSUPPORTED"),
    (dict(t=1 << 29), "UNSUPPORTED"), (dict(t=1 << 24, b=9, hq=32, width=1 << 26, stride=1 << 26, q_stride=4096), "UNSUPPORTED"),
    (dict(q=264), "ALIGNMENT"), (dict(q_stride=516), "ALIGNMENT"), (dict(lens=258), "ALIGNMENT"),
    (dict(parents=258), "ALIGNMENT")])
def test_refusals(kw, name):
    assert _abi.STATUS_NAMES[_run(**kw)] == "TA_ERR_" + name
    assert _abi.load_library().tree_attn_last_error()


def test_outputs_off_32_bytes_are_refused():
    assert _abi.STATUS_NAMES[_run(out=272)] == "TA_ERR_ALIGNMENT"  # (rows are written 32 bytes at a time)


def test_tables_of_nearly_2_31_tokens_are_refused():
    # the last step's keys, 128 and its pages' more, must be countable in 32 bits
    assert _abi.STATUS_NAMES[_run(width=(1 << 27) - 16, stride=1 << 27)] == "TA_ERR_UNSUPPORTED"


def test_workspace_of_nothing():
    f, n = _abi.load_library().tree_attn_chunk_workspace, ctypes.c_size_t(0)
    assert f(0, 0, 8, 2, 128, ctypes.byref(n)) == _abi.TA_OK and n.value == 0
    assert f(3, 100, 8, 2, 128, ctypes.byref(n)) == _abi.TA_OK
    assert _abi.STATUS_NAMES[f(1, 1, 3, 2, 128, ctypes.byref(n))] == "TA_ERR_UNSUPPORTED"
    assert _abi.STATUS_NAMES[f(1, 1, 2, 2, 128, None)] == "TA_ERR_INVALID_ARG"


def test_host_tensors_are_refused():
    for trees in (None, "mixed"):
        with pytest.raises(ValueError, match="CUDA"):
            attend(make(1, [4], None, 4, 2, 64, trees=trees))
    with pytest.raises(ValueError, match="parents"):
        s = make(1, [4], None, 4, 2, 64)
        ta.draft_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], None)


@pytest.mark.gpu
def test_wrong_tensors_are_refused():
    s = to_gpu(make(2, [4, 9], None, 4, 2, 64, trees="mixed"))
    for change in (dict(q=s["q"].half()), dict(q=s["q"].transpose(0, 1)), dict(q=s["q"][..., :32]), dict(v=s["v"][:-1]),
                   dict(table=s["table"][:1]), dict(lens=s["lens"].long()), dict(parents=s["parents"][:1]),
                   dict(parents=s["parents"].long()), dict(cu=s["lens"])):
        with pytest.raises(ValueError):
            attend({**s, **change})
    with pytest.raises(ValueError):
        attend(s, out=torch.empty(2, 4, 64, device="cuda"))
    with pytest.raises(ta.TreeAttnError):
        attend({**s, "q": s["q"][:1], "parents": s["parents"][:1]})
