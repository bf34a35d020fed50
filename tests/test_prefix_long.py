"""Attention behind long prefixes, with a bound that follows the errors' size.

Behind a long prefix an output is small (about sqrt(e / n) for n random keys),
and a bound that charges every weight's rounding at full size in one direction
is as large: it does not notice a lost key.  Here, with weights p_i, eps half a step
of the type and per row:
  - the weights' roundings, each within eps of either sign and independent:
    sum p_i d_i v_i.  By Hoeffding's inequality it passes 8 eps sqrt(sum (p_i v_i)^2)
    with a probability of 2 exp(-32) (in 10^6 elements: 3 10^-8).  fp16 adds 2^-32
    of the largest weight a key;
  - the output's own rounding, eps of it;
  - scores, off by at most X = (d + 4) 2^-24 scale max_i sum |q k_i| and by the
    exponent's own errors (3 (|s| + 1) 2^-22): sum p_i e_i (v_i - out) is at most
    X (sum p |v| + |out|);
  - sums in 32 bits over n / 16 steps, roundings of either sign: 8 sqrt(n / 16)
    2^-24 of sum p |v|, and the same of the output by the sum of weights.
The first key of every step of 128 and the last key have values 8 times as
large, so that a key or a step that goes missing at a border shows.  That it
does is tested too, on the CPU, with mistakes in the definition."""
import math

import numpy as np
import pytest
import torch

from test_prefix_attention import TYPES, attend, make, to_gpu

ta = pytest.importorskip("tree_structured_decode_gb300")

CASES = [
    # lens, queries (None: one each), heads, d, prefix
    ([100] * 40, None, (16, 4), 128, 40001),      # tiles beside the own pages, and behind them: runs of two lengths
    ([1] * 4, None, (16, 4), 128, 40001),
    ([1], None, (2, 1), 128, 20000),              # the line kernel: hundreds of runs
    ([700, 3, 2999], None, (16, 4), 64, 20000),
    ([700] * 9, None, (32, 8), 128, 12000),
    ([30] * 64, [3] * 64, (16, 2), 64, 10000),    # own tiles of 16 rows
    ([6000, 20], [2, 1], (8, 1), 128, 129),       # the own tokens are the long part
]


def case(i, dtype):
    lens, new, (hq, hkv), d, prefix = CASES[i]
    s = make(100 + i, lens, new, hq, hkv, d, prefix, dtype)
    big = [(s["pre"], prefix)] + [(s["table"][b], n) for b, n in enumerate(lens) if n >= 128]
    for pages, n in big:
        for key in {*range(0, n, 128), n - 1}:
            s["v"][pages[key // 16], :, key % 16] *= 8
    return s


def definition(s, lose=None):
    """float64 out, lse, and per row sum p |v|, sqrt(sum (p v)^2), max sum |q k|, largest p.  lose(values, scores, n): a
    mistake in the prefix's part of it, its first n keys."""
    q, k, v = (s[n].double().nan_to_num(0).numpy() for n in ("q", "k", "v"))
    t, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    got = {n: np.zeros((t, hq, d)) for n in ("out", "mean", "spread")}
    got |= {n: np.zeros((t, hq, 1)) for n in ("lse", "x", "most")}
    rows = lambda pool, pages, h, n: pool[np.asarray(pages)[: -(-n // 16)], h].reshape(-1, d)[:n]  # noqa: E731
    cu, lens = s["cu_all"], s["lens"].tolist()
    for h in range(hkv):
        kp, vp = (rows(x, s["pre"], h, s["prefix"]) for x in (k, v))
        for b, n in enumerate(lens):
            new = int(cu[b + 1]) - int(cu[b])
            at = slice(int(cu[b]), int(cu[b + 1])), slice(h * g, (h + 1) * g)
            qb = q[at].reshape(new * g, d)
            ko, vo = (rows(x, s["table"][b], h, n) for x in (k, v))
            keys, values = np.concatenate([kp, ko]), np.concatenate([vp, vo])
            score = qb @ keys.T / math.sqrt(d)
            end = len(kp) + n - new + 1 + np.repeat(np.arange(new), g)
            score[np.arange(len(keys))[None] >= end[:, None]] = -np.inf
            if lose is not None:
                values = values.copy()
                lose(values, score, len(kp))
            top = score.max(1, keepdims=True)
            w = np.exp(score - top)
            total = w.sum(1, keepdims=True)
            w /= total
            of = dict(out=w @ values, mean=w @ np.abs(values), spread=np.sqrt((w * w) @ (values * values)),
                      lse=top + np.log(total), most=w.max(1, keepdims=True),
                      x=(np.abs(qb) @ np.abs(keys).T).max(1, keepdims=True))
            for name, value in of.items():
                got[name][at] = value.reshape(new, g, -1)
    return got


def excess(s, want, out, lse):
    """How far the results pass the bound (not above 0: within it)."""
    _, eps, _ = TYPES[s["dtype"]]
    d, n = s["q"].shape[2], s["prefix"] + int(s["lens"].max())
    x = (d + 4) * 2.0 ** -24 / math.sqrt(d) * want["x"] + 3 * (np.abs(want["lse"]) + math.log(n) + 1) * 2.0 ** -22
    sums = 8 * math.sqrt(n / 16) * 2.0 ** -24
    tol = 8 * eps * want["spread"] + eps * np.abs(want["out"]) + (x + sums) * (want["mean"] + np.abs(want["out"]))
    if s["dtype"] == "fp16":
        tol += n * 2.0 ** -32 * want["most"] * 8 * np.abs(s["v"].nan_to_num(0).double().numpy()).max() + 2.0 ** -25
    over = (np.abs(out - want["out"]) - tol).max()
    return max(over, (np.abs(lse - want["lse"][..., 0]) - x[..., 0] - sums).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_definition(i, dtype):
    s = case(i, dtype)
    out, lse = attend(to_gpu(s))
    assert excess(s, definition(s), out.double().cpu().numpy(), lse.double().cpu().numpy()) <= 0


# ------------------------------------------------------------- what the bound notices (no GPU)
def last_key(values, score, n):
    score[:, n - 1] = -np.inf


def values_of_a_step(values, score, n):
    values[n // 256 * 128: n // 256 * 128 + 128] = 0


def two_values_exchanged(values, score, n):
    values[[n - 2, n - 1]] = values[[n - 1, n - 2]]


@pytest.mark.parametrize("i,dtype", [(1, "bf16"), (1, "fp16"), (2, "bf16"), (3, "fp16")])
def test_the_bound_notices_a_lost_key(i, dtype):
    s = case(i, dtype)
    kind = TYPES[dtype][0]
    want = definition(s)
    as_type = lambda x: torch.from_numpy(x).to(kind).double().numpy()  # noqa: E731
    assert excess(s, want, as_type(want["out"]), want["lse"][..., 0]) <= 0
    for lose in (last_key, values_of_a_step, two_values_exchanged):
        wrong = definition(s, lose)
        assert excess(s, want, as_type(wrong["out"]), want["lse"][..., 0]) > 0, lose.__name__
    # the lse by itself notices a lost step
    assert excess(s, want, as_type(want["out"]), want["lse"][..., 0] + math.log1p(-128 / s["prefix"])) > 0
