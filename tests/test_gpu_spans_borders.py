"""Windowed and tree attention: every key tile counts once, wherever the borders between CTAs and warps fall.

With random values a tile of a long run is lost in the bound: its weight is a few thousandths, its values have
either sign.  Here a value is 1 in one column and 0 in the others, and neighbouring tiles take neighbouring columns:
a column is then the summed weight of every d-th tile of the run, and one of them missing or counted twice
changes it by far more than its roundings (shown in test_spans_bounds; the bound is test_gpu_spans').
"""
import numpy as np
import pytest

from test_gpu_spans import Batch, built, tree_words  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

ONE = 0x3F80


def mark_tiles(b, tile, flat):
    """Token t's value: 1 in column (t // tile) % d.  flat: queries of 0, so that every key weighs the same."""
    for i, L in enumerate(b.lens):
        t = np.arange(L)
        at, off = b.tables[i][t // b.bs], t % b.bs
        b.v[at, :, off] = 0
        for h in range(b.Hkv):
            b.v[at, h, off, (t // tile + 5 * h) % b.d] = ONE
    if flat:
        b.q[:] = 0
    return b.upload()


FLAT = pytest.mark.parametrize("flat", [True, False])


@FLAT
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,chunks,Hq,Hkv", [([30000], [64], 8, 1), ([30000], [3], 2, 2), ([16384] * 3, [64] * 3, 16, 1),
                                                ([9000, 70, 20000, 700, 64, 513], [26, 8, 64, 33, 64, 1], 16, 2),
                                                ([4000, 4001, 63, 2500] * 10, [26, 1, 30, 16] * 10, 8, 2)])
def test_trees(lens, chunks, Hq, Hkv, d, flat):
    b = Batch(lens, chunks, Hq, Hkv, d, 32, seed=41)
    words = tree_words(chunks, b.rng)
    mark_tiles(b, 64, flat).tree(words)
    b.check(b.sees_tree(words))


@FLAT
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,chunks,Hq,Hkv,window,sinks",
                         [([20000], [64], 8, 1, 15000, 70), ([3000], [2500], 4, 1, 1500, 4), ([9000, 5000, 33], [40, 300, 33], 8, 2, 1 << 20, 0),
                          ([2600], [1024], 4, 4, 1000, 1), ([700, 640, 600, 655], [600] * 4, 64, 4, 640, 0),
                          ([700, 640, 600, 655], [600] * 4, 64, 4, 450, 130), ([1500] * 24, [60, 1, 128, 700] * 6, 8, 2, 1000, 4)])
def test_window_chunks(lens, chunks, Hq, Hkv, window, sinks, d, flat):
    b = Batch(lens, chunks, Hq, Hkv, d, 16, seed=42)
    mark_tiles(b, 64, flat).window(window, sinks)
    b.check(b.sees_window(window, sinks))


@FLAT
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv,window,sinks", [([30000], 8, 1, 20000, 40), ([9000, 1, 20000, 700, 0, 8192], 16, 1, 8192, 0),
                                                      ([40000, 39999], 2, 2, 1 << 20, 0), ([300, 5000, 1200, 2048, 31] * 30, 8, 2, 1024, 4),
                                                      ([129, 500] * 200, 4, 1, 128, 0), ([90, 20] * 200, 4, 1, 1 << 20, 0)])
def test_window_single_tokens(lens, Hq, Hkv, window, sinks, d, flat):
    b = Batch(lens, [1] * len(lens), Hq, Hkv, d, 16, seed=43)
    mark_tiles(b, 32, flat).window(window, sinks, single=True)
    b.check(b.sees_window(window, sinks))
