"""Scratch space of the delta rule's extend: what goes in chunks counts, and no more (no GPU needed)."""
import ctypes

import pytest

import block_sparse_attention_40_b200 as qsa
from block_sparse_attention_40_b200 import binding as B

BUDGET = 1 << 32      # above it heads run in passes


def _size(lens, heads, key_heads=None):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return qsa.load().qsa_gated_deltanet_extend_workspace_size(
        (ctypes.c_int32 * len(cu))(*cu), len(lens), key_heads or heads, heads)


@pytest.mark.parametrize("lens", [[8] * 256, [1] * 4096, [32, 0, 7], [0, 0], [1] * 65535])
def test_pieces_token_by_token_need_no_scratch(lens):
    assert _size(lens, 32) == B.WS_HEADER_BYTES


@pytest.mark.parametrize("others", [[8] * 1023, [0] * 1000, [1] * 60000, [16, 0, 3] * 300])
@pytest.mark.parametrize("lens", [[65536], [3000, 700, 8192]])
def test_short_and_empty_pieces_add_nothing(lens, others):
    assert _size(lens + others, 32) <= _size(lens, 32) + 4096
    assert _size(others + lens, 32) <= _size(lens, 32) + 4096


@pytest.mark.parametrize("lens", [[262144] + [32] * 1023, [65536] * 4, [1048576], [4096] * 500,
                                  [500000, 400000, 3, 77]])
def test_records_and_segments_stay_within_the_budget(lens):
    for heads in (2, 32, 256):
        assert 0 < _size(lens, heads) <= BUDGET + 4096, heads


def test_one_pass_where_the_used_records_fit():
    # 1,024 chunks and 1,023 short pieces: all 32 heads at once, as without the short pieces
    assert _size([65536] + [8] * 1023, 32) > 1024 * 32 * 90000
