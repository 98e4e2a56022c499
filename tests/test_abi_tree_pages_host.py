"""Which kernel a tree's call takes where the pages hold a tile of 32 keys or more (E4M3
tiles of 32 rows then take one resource), on the host (no GPU needed): the cases of
test_gpu_tree_pages.py."""

import pytest

from test_abi_attn_host import any_cache, batch
from test_abi_tree_host import KERNELS, attn_plan


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    return qlin


def table_cols(keys, page):
    return -(-keys // page)


def ordered(new, Hkv, G, tile):
    """Whether the longest sequences come first: a grid that does not fit the device at once,
    of at most 256 sequences."""
    return len(new) <= 256 and len(new) * Hkv * -(-max(new) * G // tile) > 512


@pytest.mark.parametrize("page", [32, 64, 256])
@pytest.mark.parametrize("name", KERNELS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_kernels_in_larger_pages(q, D, name, page):
    new, words, Hkv, G, keys, rows = KERNELS[name]
    i = (64, 128, 256).index(D)
    b = batch(q, batch=len(new), max_q=max(new), table_cols=table_cols(keys[i][1], page))
    got = attn_plan(q, any_cache(q, "e4m3", D, Hkv, page), b, sum(new), Hkv * G)
    assert got[0] == rows[i][1]


# Windows: new tokens of 38 sequences with 8 heads that 4 share (300 workgroups of 32 rows),
# window, keys of the table, head sizes whose E4M3 call takes 32 rows.
WINDOWS = {
    "32 rows, four waves": (100, 2048, (64,)),
    "32 rows, four waves, long": (1100, 2048, (64, 128)),
    "32 rows, eight waves": (4200, 8192, (64, 128)),
}
WINDOW_NEW, WINDOW_HKV, WINDOW_G = [8, 3, 0, 7, 8] * 7 + [5, 8, 1], 8, 4


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("name", WINDOWS)
def test_windows_in_larger_pages(q, name, page):
    window, keys, dims = WINDOWS[name]
    many = len(WINDOW_NEW) * WINDOW_HKV  # of 32 rows
    assert max(WINDOW_NEW) * WINDOW_G == 32 and 256 < many <= 512
    assert ("eight" in name) == (min(window, keys) + max(WINDOW_NEW) >= 4096)
    for D in dims:
        b = batch(q, batch=len(WINDOW_NEW), max_q=8, table_cols=table_cols(keys, page))
        got = attn_plan(q, any_cache(q, "e4m3", D, WINDOW_HKV, page), b, sum(WINDOW_NEW), WINDOW_HKV * WINDOW_G, window)
        assert got[0] == 32


# Several workgroups of 32 rows for a sequence and head, in the order of the lengths (at most
# 256 sequences) and in the batch's.
ROW_TILES = {
    "longest first": ([16, 9, 0, 13, 16, 12, 11, 10] * 8, 8, 4, 1536),
    "batch order, few at once": ([16, 9, 0, 13, 16, 12, 11, 10], 8, 4, 2 ** 16),
    "batch order, many sequences": ([16, 9, 0, 13, 16] * 60, 2, 4, 1536),
}


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("bf16", 128), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("name", ROW_TILES)
def test_row_tiles(q, name, fmt, D):
    new, Hkv, G, keys = ROW_TILES[name]
    assert max(new) * G == 64 and ordered(new, Hkv, G, 32) == ("longest" in name)
    for page in (16, 64):
        b = batch(q, batch=len(new), max_q=16, table_cols=table_cols(keys, page))
        assert attn_plan(q, any_cache(q, fmt, D, Hkv, page), b, sum(new), Hkv * G)[0] == 32, page
