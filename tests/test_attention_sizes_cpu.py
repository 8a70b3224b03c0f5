"""Workspaces of paged_attention, on the host: what a batch can need, not what the largest
could."""
import os

import pytest

import w8a8_int8_expert_amd as m

MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(m.LIB_PATH):
        from w8a8_int8_expert_amd import build
        build.build()
    return m.load_library()


def size(T, most, places, B=1, heads=32, kv_heads=8, D=128, page=64, longest=None):
    c = m.moe_w8a8_kv_cache(1000, page, kv_heads, D, m.MOE_W8A8_CACHE_BF16, None, None, 0, None,
                            None, 0)
    width = -(-places // page)
    b = m.moe_w8a8_batch(B, most, places if longest is None else longest, width, None, None, None,
                         width)
    return m.moe_w8a8_paged_attention_workspace_size(c, b, heads, T)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_that_no_piece_can_split(D):
    """A table of one piece (128 places for few rows, 512 for many) needs no room, whatever
    max_length says."""
    for T, most, B in ((40, 40, 1), (40, 40, 7), (8, 1, 8), (4000, 4000, 1)):
        assert size(T, most, 128, B=B, D=D) == 0
        assert size(T, most, 128, B=B, D=D, longest=1 << 20) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_need_what_their_rows_and_places_make(D):
    """Of each kv head: 128 rows of D + 2 values for each piece of 512 places of each row
    block, and 32 (16 of 256-wide heads) for each of 128 places of a sequence of few rows."""
    few = 16 if D == 256 else 32
    for T, places, B in ((40, 4096, 1), (64, 2000, 1), (200, 1100, 3)):
        blocks, pieces = -(-T * 4 // 128), -(-places // 512)
        part = 8 * (D + 2) * 4
        room = B * (blocks * pieces * 128 + -(-places // 128) * few) * part
        got = size(T * B, T, places, B=B, D=D)
        assert 0 < got <= room + 1024, (T, places, B)
    assert size(40, 40, 4096, D=128) < 16 * MB


def test_large_batches_need_two_rounds_of_pieces_at_most():
    cap = 8 * 130 * 4
    tiles, rows = 2 * 128 * 128 * cap, 2 * 32 * 32 * cap
    assert size(8192, 8192, 1 << 20) <= tiles + rows + 512
    assert size(8192, 8192, 1 << 20) == size(1 << 20, 1 << 20, 1 << 26, B=9)
    assert size(64, 1, 1 << 20, B=64) <= 2 * 32 * 16 * cap + 256


def test_more_places_never_need_less():
    last = 0
    for places in (64, 128, 192, 512, 576, 1024, 5000, 70000, 1 << 20):
        now = size(300, 100, places, B=3)
        assert now >= last
        last = now
