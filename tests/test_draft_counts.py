"""Counts that a kernel's 32-bit steps would run past are refused before anything is launched (no GPU)."""
import pytest

from test_drafts import _accept, _keep
from test_logprobs import _run as _scores

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("n", [MOST, MOST - 31, MOST - 128, 2 ** 30])
@pytest.mark.parametrize("call", [lambda n: _accept(t=n), lambda n: _accept(t=n, b=0), lambda n: _keep(t=n),
                                  lambda n: _scores(n_given=n), lambda n: _scores(n_given=n, rows=1)])
def test_counts_near_2_31_are_refused(call, n):
    assert _abi.STATUS_NAMES[call(n)] == "TA_ERR_UNSUPPORTED"
    assert b"2^30" in _abi.load_library().tree_attn_last_error()
