"""Many small softmax weights beside one of 1, in fp16.

Weights are rounded to the type before the product with V.  fp16 ends at 2^-24
(rounding to a multiple of it), so a weight held as 2^(s - max) would be lost
below 2^-25, and thousands of them together are more than the output's
rounding.  Held 2^7 larger, each is off by at most 2^-32 of the largest.

Bound, with n keys and |v| <= 1: n 2^-32 for these roundings, eps = 2^-11 of
the output for its own (2^-25 where it is subnormal) and of the weights' mean for
those that are normal, 2^-17 of it for the exponents (arguments up to 26 in 32
bits, exp2 to 2^-22).  The sum of weights takes a step of 16 or 128 keys at a
time: each addition is off by at most 2^-24 of it, and all in one direction,
since the small weights are equal; that is `steps` 2^-24 of the sum, and so of lse
(and of the output).  lse's own parts, up to 26 in 32 bits and rounded four times
(score, maximum, sum with the logarithm, product with ln 2): 4 * 2^-24 * 26 ln 2 <
2^-17.8, with log2 to one more step 2^-17."""
import math

import pytest
import torch

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu

TOP = 17.6875  # exact in fp16; exp(-TOP) = 2^-25.52


def pools(hkv, d):
    """Page 0 starts with the key of score TOP and value 0; page 1 and the rest of page 0 have score 0 and value 1."""
    k = torch.zeros((2, hkv, 16, d), dtype=torch.float16, device="cuda")
    v = torch.ones_like(k)
    k[0, :, 0, 0] = TOP
    v[0, :, 0] = 0
    return k, v


def check(out, lse, n, step):
    tail = (n - 1) * math.exp(-TOP)
    want = tail / (1 + tail)
    sums = -(-n // step) * 2.0 ** -24
    tol = n * 2.0 ** -32 + 2 * 2.0 ** -11 * want + 2.0 ** -25 + (2.0 ** -17 + sums) * want
    assert (out.double() - want).abs().max().item() <= tol
    assert (lse.double() - TOP - math.log1p(tail)).abs().max().item() <= 2.0 ** -17 + sums


def test_behind_a_prefix():
    """608 queries of 64 heads: 152 segments, so that each CTA's tiles go over most of the prefix."""
    k, v = pools(8, 64)
    q = torch.zeros((608, 64, 64), dtype=torch.float16, device="cuda")
    q[..., 0] = 1
    n = 30000
    pages = torch.ones(n // 16, dtype=torch.int32, device="cuda")
    pages[0] = 0
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = ta.prefix_attention(q, k, v, ints([[0]]), ints([0]), ints([0, 608]), pages, n, softmax_scale=1.0)
    check(out, lse, n, 128)


@pytest.mark.parametrize("heads", [1, 12])  # row tiles of 8 and 16
def test_a_request_s_own_tokens(heads):
    k, v = pools(1, 128)
    q = torch.zeros((2000, heads, 128), dtype=torch.float16, device="cuda")
    q[..., 0] = 1
    table = torch.ones((2000, 125), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    lens = torch.full((2000,), 2000, dtype=torch.int32, device="cuda")
    out, lse = ta.prefix_attention(q, k, v, table, lens, softmax_scale=1.0)
    check(out, lse, 2000, 16)
