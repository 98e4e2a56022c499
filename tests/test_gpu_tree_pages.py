"""Attention of trees over pages that hold a tile of 32 keys or more, on the GPU against the
fp64 oracle: E4M3 tiles of 32 rows take one resource there. Which kernel a case runs is
pinned in test_abi_tree_pages_host.py. Bounds as in the tests of attention (attn_check)."""

import numpy as np
import pytest
import torch

from test_abi_tree_host import KERNELS
from test_abi_tree_pages_host import ROW_TILES, WINDOW_G, WINDOW_HKV, WINDOW_NEW, WINDOWS, table_cols
from test_gpu_tree import run_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_linear_layers_amd as qlin

    assert torch.cuda.is_available()
    return qlin


def to_width(keys, page, kv):
    """Columns behind the sequences' own that make the table as wide as the case's."""
    return table_cols(keys, page) - max(-(-k // page) for k in kv)


@pytest.mark.parametrize("page", [32, 64, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", KERNELS)
def test_kernels_in_larger_pages(q, oracle, name, D, page):
    new, words, Hkv, G, keys, _ = KERNELS[name]
    keys = keys[(64, 128, 256).index(D)][1]
    rng = np.random.default_rng(D + page)
    kv = [n + int(rng.integers(0, min(keys, 500) - 16 * words)) for n in new]
    if keys > 1024:
        kv[0] = new[0] + 1000
    run_tree(q, oracle, D + page, new, kv, Hkv, G, D, page, "e4m3", words=words, extra_cols=to_width(keys, page, kv), pad=1)


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("name,D", [(name, D) for name in WINDOWS for D in WINDOWS[name][2]])
def test_windows_in_larger_pages(q, oracle, name, D, page):
    """The first seen key at every place in a tile and a page: rows before it are not read."""
    window, keys, _ = WINDOWS[name]
    rng = np.random.default_rng(window + D)
    kv = [n + int(rng.integers(0, 200)) for n in WINDOW_NEW]
    for b in range(0, len(kv), 2 if window <= 1100 else 12):
        kv[b] = WINDOW_NEW[b] + window + int(rng.integers(0, 90))

    def edit(rng, mask, pos):  # positions before the first and behind the last token: the nearest of those
        pos[1], pos[30], pos[31] = -5, 2 ** 31 - 1, 0

    run_tree(q, oracle, D, WINDOW_NEW, kv, WINDOW_HKV, WINDOW_G, D, page, "e4m3", window=window,
             extra_cols=to_width(keys, page, kv), edit=edit)


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", ["32 rows, eight waves", "32 rows, four waves"])
def test_missing_pages_and_short_sequences_in_larger_pages(q, oracle, name, D, page):
    """Pages that do not exist among earlier and new tokens, fewer cached keys than new
    tokens, none, masks that are no trees."""
    new, words, Hkv, G, keys, _ = KERNELS[name]
    keys = keys[(64, 128).index(D)][1]
    rng = np.random.default_rng(D + page)
    kv = [n + int(rng.integers(0, 500)) for n in new]
    kv[0], kv[1], kv[3] = 16 + 700, 4, 0

    def pages(table):
        table[0, [0, 3, 700 // page]] = -1, 10 ** 9, -1
        table[4:, 1] = 2 ** 31 - 1  # (some sequences end before it)

    def masks(rng, mask, pos):
        mask[:16] = rng.integers(0, 2 ** 64, mask[:16].shape, dtype=np.uint64)
        mask[2], mask[20] = 0, 0

    r = run_tree(q, oracle, D + page, new, kv, Hkv, G, D, page, "e4m3", words=words,
                 extra_cols=to_width(keys, page, kv), table_edit=pages, edit=masks, pad=2)
    assert (r["seen"][25:38] == 0).all() and (r["seen"][20] == 0).all()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("bf16", 128), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("name", ROW_TILES)
def test_row_tiles(q, oracle, name, fmt, D, page):
    """Ragged sequences of up to two workgroups' rows, some without new tokens, some as long
    as others, in the order of their lengths and in the batch's."""
    new, Hkv, G, keys = ROW_TILES[name]
    rng = np.random.default_rng(D + page)
    kv = [n + int(rng.choice([0, 7, 100, 100, 350])) for n in new]
    kv[len(kv) // 2] = new[len(kv) // 2] + 1200
    run_tree(q, oracle, D + page, new, kv, Hkv, G, D, page, fmt, extra_cols=to_width(keys, page, kv), pad=1)
