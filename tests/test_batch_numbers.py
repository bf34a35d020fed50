"""Numbers that do not fit the C ABI's 32 bits are refused, not cut."""
import os
import re

import pytest
import torch

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi, batch  # noqa: E402

TOO_LARGE = [2 ** 31, 2 ** 32 + 5, 2 ** 63, -2 ** 31 - 1, -2 ** 32 + 5]


@pytest.mark.parametrize("x", TOO_LARGE)
def test_extension(x):
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_new"):
        ta.extend_tables(z, z, z.reshape(1, 1), z, z, x)
    with pytest.raises(ValueError, match="position_base"):
        ta.extend_tables(z, z, z.reshape(1, 1), z, z, 1, position_base=x)


@pytest.mark.parametrize("x", TOO_LARGE)
def test_prefix_length(x):
    z = torch.zeros(1, dtype=torch.int32)
    pool = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="prefix_len"):
        ta.prefix_attention(pool[0, :, 0].reshape(1, 1, 64), pool, pool, z.reshape(1, 1), z, None, z, x)


def test_tensors_of_too_many_entries():
    """(Tensors without memory.)"""
    z = torch.zeros(1, dtype=torch.int32)
    wide = torch.empty((1, 2 ** 32 + 4), dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        batch._table(wide, 1, -1, torch.int32)
    with pytest.raises(ValueError, match="free_pages.*32 bits"):
        ta.extend_tables(z, z, z.reshape(1, 1), wide[0], z, 1)
    with pytest.raises(ValueError, match="lens.*32 bits"):
        ta.extend_tables(wide[0], wide[0], z.reshape(1, 1), z, z, 1)
    with pytest.raises(ValueError, match="32 bits"):
        ta.sample(torch.empty((2 ** 32 + 1, 1), device="meta"), torch.empty((2 ** 32 + 1,), device="meta"))


def test_limits_and_bits_are_the_header_s():
    path = os.path.join(os.path.dirname(__file__), "..", "include", "tree_attn.h")
    with open(path) as f:
        said = dict(re.findall(r"TREE_ATTN_(MAX_\w+|BATCH_\w+) =? ?(\d+)", f.read()))
    assert len(said) == 7
    for name, value in said.items():
        assert getattr(_abi, name) == int(value), name
