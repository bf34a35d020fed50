"""Temperatures up to +inf: every logit above -inf has the same weight there, masked ones keep -inf.
Tolerances: test_logprobs.py; with T above 2^126 the factor 1 / T is subnormal, a multiple of 2^-149, so y = (x - max) / T
is off by at most 2^-150 |x - max|: with |x - max| < 2^128 by 2^-22, less than the bound's 2^-20."""
import math

import pytest
import torch

from test_logprobs import check, logits, run

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heat", [1e30, 1e38, 2e38, 3.4e38, 1e39, math.inf])
@pytest.mark.parametrize("vocab", [40, 3001, 150000])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masked_tokens_stay_masked(dtype, vocab, heat):
    x = logits(vocab, 6, vocab, dtype)
    lowest = torch.finfo(x.dtype).min
    x[1, 1::2] = -math.inf
    x[2, 1:] = -math.inf
    x[3, 1::2] = lowest             # a mask's lowest value is a logit like others
    x[4] = lowest
    x[4, 3] = -math.inf
    x[5, 1] = math.inf
    given = [[0, 1, 3, vocab - 1, -1]] * 6
    for top in (0, 5):
        check(x, given, heat, top, run(x, given, heat, top))
        check(x, given, [heat] * 6, top, run(x, given, [heat] * 6, top))
