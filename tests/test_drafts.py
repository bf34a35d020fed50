"""Accepted drafts and the move of their keys and values, against their
definitions; results are whole numbers and copies, equal bit for bit."""
import numpy as np
import pytest
import torch

from oracle import drafts as oracle
from test_chunk_attention import tree

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402

ints = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731


def batch(seed, counts, kind="mixed", vocab=6, padding=3):
    """Trees over a small vocabulary, so that siblings share tokens and paths are long; some nodes drew nothing (-1)."""
    g = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    parents = sum((tree(seed + b, n, kind) for b, n in enumerate(counts)), []) + [3] * padding
    t = len(parents)
    return dict(drafted=g.integers(0, vocab, t).tolist(), parents=parents, cu=cu.tolist(),
                sampled=np.where(g.random(t) < 0.05, -1, g.integers(0, vocab, t)).tolist())


def accept(s, **kw):
    c = {n: ints(x).cuda() for n, x in s.items()}
    return ta.accept_drafts(c["drafted"], c["parents"], c["cu"], c["sampled"], **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,vocab", [("mixed", 6), ("mixed", 2), ("chain", 2), ("star", 40), ("roots", 2), ("chain", 1)])
@pytest.mark.parametrize("counts", [[1], [0], [128], [5, 0, 64, 1, 33, 32, 0], [127] * 20, [7] * 300])
def test_accepted_paths(counts, kind, vocab):
    s = batch(len(counts) + vocab, counts, kind, vocab)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = accept(s, status=status)
    assert [x.tolist() for x in got] == list(oracle.accept_drafts(**s)) and status.item() == 0


@pytest.mark.gpu
def test_drafts_that_are_none():
    """Drafted tokens below 0 match nothing, not even a node that drew nothing."""
    got = accept(dict(drafted=[4, -1, 3], parents=[-1, 0, 0], cu=[0, 3], sampled=[-1, 3, 3]))
    assert [x.tolist() for x in got] == [[0, -1, -1], [1], [-1], [-2]]


@pytest.mark.gpu
def test_bad_trees_and_offsets():
    def run(**kw):
        s = batch(4, [6, 129, 5], vocab=2, padding=0)
        s.update(kw)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s, [x.tolist() for x in accept(s, status=status)], status.item()

    s, got, status = run()
    assert status == _abi.BATCH_BAD_INPUT  # 129 nodes: none is kept
    path, kept, following, back = oracle.accept_drafts(**s)
    assert got[0] == path[:6] + [-1] * 129 + path[135:]
    assert got[1:] == [[kept[0], 0, kept[2]], [following[0], -1, following[2]], [back[0], -129, back[2]]]
    for cu in ([0, 140, 141, 141], [0, 6, 5, 140], [-1, 6, 20, 30], [0, 2, 3, -4]):
        _, got, status = run(cu=cu)
        assert status == _abi.BATCH_BAD_INPUT and got == [[-1] * 140, [0] * 3, [-1] * 3, [0] * 3]
    _, got, _ = run(cu=[3, 5, 5, 9])  # tokens before the first request's (whose parents are then another's)
    assert got[0][:3] == [-1] * 3 and got[0][9:] == [-1] * 131
    s = dict(drafted=[1, 1, 1, 1], parents=[-1, 0, 2, 99], cu=[0, 4], sampled=[1, 1, 1, 1])  # itself, far above
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert [x.tolist() for x in accept(s, status=status)] == [[0, 1, -1, -1], [2], [1], [-2]]
    assert status.item() == _abi.BATCH_BAD_INPUT


def cache(seed, counts, held, layers, hkv, d, kind=torch.bfloat16):
    """Bits of pools and shuffled tables."""
    g = torch.Generator().manual_seed(seed)
    lens = [h + n for h, n in zip(held, counts)]
    width = max([1] + [-(-n // 16) for n in lens])
    total = sum(-(-n // 16) for n in lens) + 1
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for j in range(-(-n // 16)):
            table[b, j] = order.pop()
    pool = lambda: torch.randint(-2 ** 15, 2 ** 15, (layers, total, hkv, 16, d), generator=g, dtype=torch.int16)  # noqa: E731
    return dict(table=table, lens=ints(lens), k=pool(), v=pool())


@pytest.mark.gpu
@pytest.mark.parametrize("counts,held,layers,hkv,d", [
    ([1], [0], 1, 1, 64), ([8, 0, 5], [3, 16, 30], 1, 4, 64), ([60] * 5, [0, 1, 15, 16, 100], 3, 2, 128),
    ([128, 127], [9, 40], 2, 5, 64), ([6] * 40, [20] * 40, 5, 8, 128)])
@pytest.mark.parametrize("kind,vocab", [("mixed", 2), ("chain", 2), ("star", 3)])
def test_moves(counts, held, layers, hkv, d, kind, vocab):
    s = batch(sum(counts), counts, kind, vocab)
    c = cache(7, counts, held, layers, hkv, d)
    path, *_ = oracle.accept_drafts(**s)
    k, v = (c[n].cuda().view(torch.bfloat16) for n in "kv")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ta.keep_drafts(ints(path).cuda(), ints(s["cu"]).cuda(), c["table"].cuda(), c["lens"].cuda(), k, v, status=status)
    want = oracle.keep_drafts(path, s["cu"], c["table"].numpy(), c["lens"].numpy(), c["k"].numpy(), c["v"].numpy())
    assert status.item() == 0
    assert np.array_equal(k.view(torch.int16).cpu().numpy(), want[0]) and np.array_equal(v.view(torch.int16).cpu().numpy(), want[1])


@pytest.mark.gpu
def test_long_paths_and_pools_apart():
    """A path of every second of 700 nodes (moves by the hundred, sources that are targets too), layers with room between
    them, a pool of one layer given as such."""
    path = list(range(0, 700, 2)) + [-1] * 350
    c = cache(3, [700], [21], 3, 2, 64)
    apart = torch.zeros((3, c["k"].shape[1] + 2, 2, 16, 64), dtype=torch.int16)
    k, v = apart.clone().cuda(), apart.clone().cuda()
    k[:, :-2], v[:, :-2] = c["k"].cuda(), c["v"].cuda()
    pools = [x.view(torch.bfloat16)[:, :-2] for x in (k, v)]
    args = ints(path).cuda(), ints([0, 700]).cuda(), c["table"].cuda(), c["lens"].cuda()
    ta.keep_drafts(*args, *pools)
    want = oracle.keep_drafts(path, [0, 700], c["table"].numpy(), c["lens"].numpy(), c["k"].numpy(), c["v"].numpy())
    for got, was in zip((k, v), want):
        assert np.array_equal(got[:, :-2].cpu().numpy(), was) and not got[:, -2:].any()
    one = [c[n][1].cuda().view(torch.bfloat16) for n in "kv"]
    ta.keep_drafts(*args, *one)
    for got, was in zip(one, want):
        assert np.array_equal(got.view(torch.int16).cpu().numpy(), was[1])


@pytest.mark.gpu
def test_bad_paths_stay_in_bounds():
    counts, held = [8, 6], [10, 5]
    for name, at, value, bit, moved in (
            ("path", 2, 8, _abi.BATCH_BAD_INPUT, [0, 3, -1]), ("path", 2, 3, _abi.BATCH_BAD_INPUT, [0, 3, -1]),
            ("path", 1, -9, _abi.BATCH_BAD_INPUT, [0, -1]), ("path", 0, -3, _abi.BATCH_BAD_INPUT, [-1]),
            ("table", (0, 1), 99, _abi.BATCH_BAD_SLOT, [0, 3, -1]),
            ("table", (0, 1), -1, _abi.BATCH_BAD_SLOT, [0, 3, -1]), ("lens", 0, 7, _abi.BATCH_BAD_INPUT, [-1]),
            ("lens", 0, 10 ** 6, _abi.BATCH_BAD_INPUT, [-1]), ("cu", 1, 50, _abi.BATCH_BAD_INPUT, None)):
        c = cache(5, counts, held, 1, 2, 64)
        c.update(path=ints([0, 3, 6, 7, -1, -1, -1, -1, 0, 2, -1, 5, 5, 5]), cu=ints([0, 8, 14]))
        good = {n: x.clone() for n, x in c.items()}
        c[name][at] = value
        k, v = (c[n].cuda().view(torch.bfloat16) for n in "kv")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ta.keep_drafts(*(c[n].cuda() for n in ("path", "cu", "table", "lens")), k, v, status=status)
        assert status.item() == bit
        if moved is None:
            assert torch.equal(k.view(torch.int16).cpu(), c["k"])
            continue
        path = moved + [-1] * (8 - len(moved)) + [0, 2, -1] + [-1] * 3
        want = oracle.keep_drafts(path, [0, 8, 14], good["table"].numpy(), good["lens"].numpy(), c["k"].numpy(), c["v"].numpy())
        assert np.array_equal(k.view(torch.int16).cpu().numpy(), want[0]) and np.array_equal(v.view(torch.int16).cpu().numpy(), want[1])


@pytest.mark.gpu
def test_nothing_to_do():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert [x.numel() for x in ta.accept_drafts(z, z, cu, z)] == [0, 0, 0, 0]
    got = ta.accept_drafts(*[torch.ones(3, dtype=torch.int32, device="cuda")] * 2, cu, torch.ones(3, dtype=torch.int32, device="cuda"))
    assert got[0].tolist() == [-1] * 3
    pool = torch.ones((2, 1, 16, 64), dtype=torch.float16, device="cuda")
    ta.keep_drafts(z, cu, z.reshape(0, 1), z, pool, pool)
    ta.keep_drafts(z, torch.zeros(2, dtype=torch.int32, device="cuda"), cu.reshape(1, 1), cu, pool[None][:0], pool[None][:0])


# ------------------------------------------------------------- refusals (no GPU)
def _accept(**kw):
    a = dict(drafted=256, parents=256, cu=256, sampled=256, b=2, t=5, path=256, kept=256, next=256, back=256, status=None,
             stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_accept_drafts(*a.values())


def _keep(**kw):
    a = dict(path=256, cu=256, lens=256, table=256, stride=4, width=4, b=2, t=5, k=256, v=256, between=0, layers=2, pages=9,
             hkv=2, d=128, status=None, stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_keep_drafts(*a.values())


@pytest.mark.parametrize("f,kw,name", [
    (_accept, dict(drafted=None), "INVALID_ARG"), (_accept, dict(parents=None), "INVALID_ARG"),
    (_accept, dict(sampled=None), "INVALID_ARG"), (_accept, dict(path=None), "INVALID_ARG"),
    (_accept, dict(kept=None), "INVALID_ARG"), (_accept, dict(next=None), "INVALID_ARG"),
    (_accept, dict(b=-1), "INVALID_ARG"), (_accept, dict(t=-1), "INVALID_ARG"), (_accept, dict(cu=None), "INVALID_ARG"),
    (_accept, dict(b=16385), "UNSUPPORTED"), (_accept, dict(back=257), "ALIGNMENT"),
    (_keep, dict(path=None), "INVALID_ARG"), (_keep, dict(lens=None), "INVALID_ARG"), (_keep, dict(table=None), "INVALID_ARG"),
    (_keep, dict(k=None), "INVALID_ARG"), (_keep, dict(b=-1), "INVALID_ARG"), (_keep, dict(stride=3), "INVALID_ARG"),
    (_keep, dict(cu=None), "INVALID_ARG"), (_keep, dict(between=8), "INVALID_ARG"), (_keep, dict(layers=-1), "INVALID_ARG"),
    (_keep, dict(hkv=0), "INVALID_ARG"), (_keep, dict(d=80), "UNSUPPORTED"), (_keep, dict(layers=1 << 16), "UNSUPPORTED"),
    (_keep, dict(b=16385), "UNSUPPORTED"), (_keep, dict(pages=(1 << 27) + 1), "UNSUPPORTED"),
    (_keep, dict(between=(1 << 20) + 4), "ALIGNMENT"), (_keep, dict(v=264), "ALIGNMENT"), (_keep, dict(cu=258), "ALIGNMENT")])
def test_refusals(f, kw, name):
    assert _abi.STATUS_NAMES[f(**kw)] == "TA_ERR_" + name
    assert _abi.load_library().tree_attn_last_error()


def test_limits_are_the_header_s():
    import os
    import re

    with open(os.path.join(os.path.dirname(__file__), "..", "include", "tree_attn.h")) as f:
        said = dict(re.findall(r"#define TREE_ATTN_(\w+_MAX) (\d+)", f.read()))
    assert said and all(getattr(_abi, name) == int(value) for name, value in said.items())


def test_wrong_tensors_are_refused():
    z, cu = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ta.accept_drafts(z, z, cu, z)
    with pytest.raises(ValueError, match="CUDA"):
        ta.keep_drafts(z, cu, cu.reshape(1, 2), cu[:1], pool, pool)


@pytest.mark.gpu
def test_wrong_cuda_tensors_are_refused():
    z, cu = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    pool = torch.zeros((2, 1, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    for args in ((z, z[:2], cu, z), (z, z, cu, z.long()), (z, z, cu[:0], z), (z, z, cu.cpu(), z)):
        with pytest.raises(ValueError):
            ta.accept_drafts(*args)
    table, lens = cu.reshape(1, 2), cu[:1]
    for args in ((z, cu[:1], table, lens, pool, pool), (z, cu, table, lens, pool, pool[:1]), (z, cu, z.reshape(3, 1), lens, pool, pool),
                 (z, cu, table, lens, pool.float(), pool.float()), (z, cu, table, lens, pool[..., :32], pool[..., :32]),
                 (z.long(), cu, table, lens, pool, pool), (z, cu, table, lens, pool[:1].expand(2, 1, 1, 16, 64), pool[:1].expand(2, 1, 1, 16, 64)),
                 (z, cu, table, lens, pool.expand(2, 2, 1, 16, 64).transpose(0, 1), pool.expand(2, 2, 1, 16, 64).transpose(0, 1))):
        with pytest.raises((ValueError, ta.TreeAttnError)):
            ta.keep_drafts(*args)
