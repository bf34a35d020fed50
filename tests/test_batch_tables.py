"""Page tables and slot maps built on the GPU, and the append by slot, against
their definitions in Python integers.  Everything here is whole numbers or
copies: results are equal, not close."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import batch as oracle

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402


def _state(seed, requests, width, capacity, held, device="cuda"):
    """Random requests holding up to `held` tokens each, and the stack of the other pages."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, held + 1, size=requests)
    pages = rng.permutation(capacity).tolist()
    table = np.full((requests, width), -7)
    for b, n in enumerate(lens):
        for j in range(-(-int(n) // 16)):
            table[b, j] = pages.pop()
    free = np.array(pages + [-9] * (capacity - len(pages)))
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    return rng, put(lens), put(table), put(free), put([len(pages)])


def _check(lens, n_new, table, free, n_free, max_new, base=0, status=None):
    want = oracle.extend_tables(lens.tolist(), n_new.tolist(), table.tolist(), free.tolist(), n_free.item(), max_new, base)
    slots, positions, cu = ta.extend_tables(lens, n_new, table, free, n_free, max_new, position_base=base, status=status)
    assert want is not None
    for name, got, w in zip(("slots", "positions", "cu", "lens", "table", "free", "n_free"),
                            (slots, positions, cu, lens, table, free, n_free), want):
        assert got.tolist() == (w if name != "n_free" else [w]), name
    return slots, positions, cu


@pytest.mark.gpu
@pytest.mark.parametrize("requests,held,new", [(1, 0, 1), (1, 15, 1), (1, 16, 1), (3, 40, 5), (64, 200, 1), (64, 100, 90),
                                               (257, 33, 20), (1025, 17, 4), (2500, 30, 3), (16384, 20, 2)])
def test_extend_and_take_back(requests, held, new):
    width = -(-(held + 3 * new) // 16) + 1
    rng, lens, table, free, n_free = _state(requests + held, requests, width, requests * width + 3, held)
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    status = put([0])
    before = [x.clone() for x in (lens, free, n_free)]
    n = put(rng.integers(0, new + 1, size=requests))
    _check(lens, n, table, free, n_free, requests * new + 5, base=11, status=status)
    _check(lens, -n, table, free, n_free, 0, status=status)
    # an extension taken back leaves lengths and stack as they were
    for a, b in zip(before, (lens, free, n_free)):
        assert torch.equal(a, b)
    # some grow, some shrink, some end (more taken back than they hold)
    n = put(rng.integers(-held - 40, new + 1, size=requests))
    _check(lens, n, table, free, n_free, requests * new, status=status)
    _check(lens, put(rng.integers(-20, new + 1, size=requests)), table, free, n_free, requests * new, base=5, status=status)
    assert status.item() == 0


@pytest.mark.gpu
def test_build_from_nothing_in_a_wide_table_view():
    rng, lens, _, free, n_free = _state(5, 40, 1, 40 * 70, 0)
    wide = torch.full((40, 100), -3, dtype=torch.int32, device="cuda")
    n = torch.tensor(rng.integers(1, 1024, size=40), dtype=torch.int32, device="cuda")
    _check(lens, n, wide[:, 5:70], free, n_free, 40 * 1024)
    assert (wide[:, :5] == -3).all() and (wide[:, 70:] == -3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("what,bit", [("pages", "BATCH_NO_PAGES"), ("row", "BATCH_TABLE_FULL"), ("outputs", "BATCH_TABLE_FULL"),
                                      ("length", "BATCH_BAD_INPUT"), ("long", "BATCH_BAD_INPUT"), ("stack", "BATCH_BAD_INPUT"),
                                      ("deep", "BATCH_BAD_INPUT"), ("overflow", "BATCH_BAD_INPUT")])
def test_all_or_nothing(what, bit):
    _, lens, table, free, n_free = _state(9, 30, 6, 200, 50)
    n = torch.full((30,), 10, dtype=torch.int32, device="cuda")
    most, status = 300, torch.tensor([0], dtype=torch.int32, device="cuda")
    if what == "pages":
        n_free.fill_(4)
    elif what == "row":
        n[7] = 97
    elif what == "outputs":
        most = 299
    elif what == "length":
        lens[3] = -1
    elif what == "long":
        lens[3] = 97
    elif what == "stack":
        n_free.fill_(201)
    elif what == "deep":
        n_free.fill_(-1)
    else:  # more pages given back than the stack has room for
        n_free.fill_(200)
        n.fill_(-60)
    before = [x.clone() for x in (lens, table, free, n_free)]
    slots, positions, cu = ta.extend_tables(lens, n, table, free, n_free, most, status=status)
    assert status.item() == getattr(_abi, bit)
    for a, b in zip(before, (lens, table, free, n_free)):
        assert torch.equal(a, b)
    assert (slots == -1).all() and (positions == -1).all() and (cu == 0).all()
    # without a status word as well
    ta.extend_tables(lens, n, table, free, n_free, most)


@pytest.mark.gpu
def test_no_request_and_no_new_token():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    free, n_free = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32, device="cuda")
    slots, positions, cu = ta.extend_tables(z, z, torch.zeros((0, 3), dtype=torch.int32, device="cuda"), free, n_free, 3)
    assert slots.tolist() == [-1] * 3 and cu.tolist() == [0] and n_free.item() == 4
    _, lens, table, free, n_free = _state(1, 5, 4, 30, 40)
    _check(lens, torch.zeros_like(lens), table, free, n_free, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hkv,d", [(1, 1, 64), (7, 3, 128), (300, 8, 128), (65, 40, 64), (33, 17, 128)])
def test_append_by_slot(tokens, hkv, d, dtype):
    g = torch.Generator().manual_seed(tokens)
    pages = tokens // 8 + 2
    pool = lambda: torch.randn((pages, hkv, 16, d), generator=g).to(dtype)  # noqa: E731
    k, v = pool(), pool()
    joint = torch.randn((tokens, 2 * hkv + 3, d), generator=g).to(dtype)
    slots = torch.randperm(pages * 16, generator=g)[:tokens].to(torch.int32)
    slots[tokens // 2] = -1
    if tokens > 10:
        slots[3], slots[9] = pages * 16, -5  # outside: skipped, and said so
    bits = lambda x: x.view(torch.int16).cpu().numpy()  # noqa: E731
    want = oracle.append_slots(bits(joint[:, :hkv].contiguous()), bits(joint[:, hkv:2 * hkv].contiguous()), slots, bits(k), bits(v))
    j, kc, vc, status = joint.cuda(), k.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    ta.append_slots(j[:, :hkv], j[:, hkv:2 * hkv], slots.cuda(), kc, vc, status=status)
    assert np.array_equal(bits(kc), want[0]) and np.array_equal(bits(vc), want[1])
    assert status.item() == (_abi.BATCH_BAD_SLOT if tokens > 10 else 0)


@pytest.mark.gpu
def test_captured_steps_advance_the_state():
    """One captured step, replayed: lengths, tables and slots go on from step to step, on another stream than the current."""
    rng, lens, table, free, n_free = _state(21, 20, 12, 400, 30)
    state = [x.clone() for x in (lens, table, free, n_free)]
    n = torch.tensor(rng.integers(0, 4, size=20), dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = ta.extend_tables(lens, n, table, free, n_free, 80, position_base=2)
    for _ in range(6):
        want = oracle.extend_tables(state[0].tolist(), n.tolist(), state[1].tolist(), state[2].tolist(), state[3].item(), 80, 2)
        graph.replay()
        torch.cuda.synchronize()
        assert [x.tolist() for x in out] == list(want[:3])
        state = [torch.tensor(x, dtype=torch.int32) for x in (*want[3:6], [want[6]])]
        for a, b in zip(state, (lens, table, free, n_free)):
            assert torch.equal(a, b.cpu())


@pytest.mark.gpu
def test_a_stream_that_is_given():
    _, lens, table, free, n_free = _state(3, 9, 8, 90, 30)
    stream = torch.cuda.Stream()
    n = torch.full((9,), 3, dtype=torch.int32, device="cuda")
    want = oracle.extend_tables(lens.tolist(), n.tolist(), table.tolist(), free.tolist(), n_free.item(), 27)
    torch.cuda.synchronize()
    out = ta.extend_tables(lens, n, table, free, n_free, 27, stream=stream)
    again = ta.extend_tables(lens, -n, table, free, n_free, 0, stream=stream.cuda_stream)
    stream.synchronize()
    assert [x.tolist() for x in out] == list(want[:3]) and again[0].numel() == 0


# ------------------------------------------------------------- refusals (no GPU)
def _extend(**kw):
    a = dict(lens=64, n_new=64, n_requests=2, table=64, stride=4, width=4, free=64, cap=8, n_free=64, max_new=2, base=0,
             slots=64, positions=64, cu=64, status=None, stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_extend_tables(*a.values())


@pytest.mark.parametrize("kw,name", [
    (dict(n_requests=-1), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"), (dict(n_new=None), "INVALID_ARG"),
    (dict(table=None), "INVALID_ARG"), (dict(stride=3), "INVALID_ARG"), (dict(free=None), "INVALID_ARG"),
    (dict(n_free=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"), (dict(positions=None), "INVALID_ARG"),
    (dict(max_new=-1), "INVALID_ARG"), (dict(base=-1), "INVALID_ARG"), (dict(cap=-1), "INVALID_ARG"),
    (dict(n_requests=16385), "UNSUPPORTED"), (dict(width=1 << 27, stride=1 << 27), "UNSUPPORTED"),
    (dict(lens=66), "ALIGNMENT"), (dict(cu=65), "ALIGNMENT"), (dict(status=2), "ALIGNMENT")])
def test_extend_refusals(kw, name):
    assert _abi.STATUS_NAMES[_extend(**kw)] == "TA_ERR_" + name
    assert _abi.load_library().tree_attn_last_error()


def _append(**kw):
    a = dict(k_new=64, v_new=64, ks=128, vs=128, slots=64, tokens=2, hkv=1, d=128, k=64, v=64, pages=4, status=None, stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_append_slots(*a.values())


@pytest.mark.parametrize("kw,name", [
    (dict(k_new=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"),
    (dict(tokens=-1), "INVALID_ARG"), (dict(hkv=0), "INVALID_ARG"), (dict(pages=-1), "INVALID_ARG"),
    (dict(ks=120), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"), (dict(hkv=5000), "UNSUPPORTED"),
    (dict(pages=(1 << 27) + 1), "UNSUPPORTED"), (dict(k_new=72), "ALIGNMENT"), (dict(vs=132), "ALIGNMENT"),
    (dict(slots=66), "ALIGNMENT")])
def test_append_refusals(kw, name):
    assert _abi.STATUS_NAMES[_append(**kw)] == "TA_ERR_" + name


def test_append_of_no_token_is_done_at_once():
    assert _append(tokens=0) == _abi.TA_OK


def test_host_tensors_are_refused():
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ta.extend_tables(z, z, z.reshape(1, 1), z, z, 1)
    x = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ta.append_slots(x[0], x[0], z, x, x)


@pytest.mark.gpu
def test_wrong_tensors_are_refused():
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    one, table = z[:1], torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for bad in (lambda: ta.extend_tables(z.long(), z, table, z, one, 1), lambda: ta.extend_tables(z, z[:3], table, z, one, 1),
                lambda: ta.extend_tables(z, z, table[:3], z, one, 1), lambda: ta.extend_tables(z, z, table.t(), z, one, 1),
                lambda: ta.extend_tables(z, z, table, z, z, 1), lambda: ta.extend_tables(z, z, table, z, one, -1),
                lambda: ta.extend_tables(z, z, table, z.cpu(), one, 1)):
        with pytest.raises(ValueError):
            bad()
    k = torch.zeros((2, 3, 16, 64), dtype=torch.bfloat16, device="cuda")
    new = torch.zeros((4, 3, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: ta.append_slots(new.half(), new, z, k, k), lambda: ta.append_slots(new[:3], new, z, k, k),
                lambda: ta.append_slots(new[:, :2], new[:, :2], z, k, k), lambda: ta.append_slots(new, new, z[:3], k, k),
                lambda: ta.append_slots(new, new, z, k.float(), k.float()),
                lambda: ta.append_slots(new.transpose(1, 2).contiguous().transpose(1, 2), new, z, k, k)):
        with pytest.raises(ValueError):
            bad()
