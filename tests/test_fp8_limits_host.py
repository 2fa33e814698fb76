"""Sizes that the fp8 attention refuses, before any CUDA call: key positions are 32-bit numbers, and the
last tile's and split's ends lie past the last key."""
import ctypes

import pytest

from test_step_host import caller, lib  # noqa: F401

INT_MAX = (1 << 31) - 1


@pytest.mark.parametrize("stride", [(1 << 30) + 1, INT_MAX - 1072, INT_MAX])
def test_table_rows_past_the_limit(lib, stride):  # noqa: F811
    P = ctypes.c_void_p
    f = caller(lib, "mla_verify_attn_fp8", q=P(16), lat=P(16), sc=P(16), rope=P(16), pool=10, table=P(16), stride=16,
               seq=P(16), mask=None, bits=None, B=1, q_len=9, H=8, scale=0.1, out=P(16), lse=P(16), ns=1, ws=None, wsb=0,
               st=None)
    assert f(stride=stride) == -2
    assert f(stride=1 << 30, q=P(24)) == -3            # the largest passes on to the next check


def test_positions_fit_up_to_the_limit():
    """split_range and the tile loop in exact integers at the limit: every intermediate fits 32 bits."""
    n, tile = 1 << 30, 48
    for S in (1, 2, 3, 152, 1023, 1024):
        assert n + S - 1 <= INT_MAX
        chunk = -(-n // S)
        assert chunk + tile - 1 <= INT_MAX
        chunk = -(-chunk // tile) * tile
        for s in (0, S // 2, S - 1):
            begin, end = min(n, s * chunk), min(n, (s + 1) * chunk)
            tiles = -(-(end - begin) // tile)
            # slots are asked for up to eight tiles ahead of the last, positions compared a tile past it
            assert begin + (tiles + 8) * tile + tile <= INT_MAX
