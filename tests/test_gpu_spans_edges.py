"""Windowed and tree attention at the ends of their integers: block ids and windows as large as their types hold."""
import numpy as np
import pytest

from oracle import spans as OS
from test_gpu_spans import Batch, bits, built, check  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

LARGEST = 2 ** 31 - 1


@pytest.mark.parametrize("bad", [-1, -(1 << 31), LARGEST, 1 << 30, "NB"])
@pytest.mark.parametrize("form", ["tree", "chunk", "single"])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 128)])
def test_bad_block_ids_are_reported_and_not_read(d, bs, form, bad):
    """The sequence's rows come out over zeros in the block's place; the other sequences are as ever."""
    c = 1 if form == "single" else 4
    words = [15] * (3 * c)
    b = Batch([600, 900, 400], [c] * 3, 4, 2, d, bs, seed=51)
    sees = b.sees_tree(words) if form == "tree" else b.sees_window(300, 2)
    e = 590 // bs  # seen by the first sequence's rows
    ref, mag, dot = b.expect(sees)
    b.upload()
    b.gt[0, e] = b.NB if bad == "NB" else bad
    if form == "tree":
        b.tree(words, 4)
    else:
        b.window(300, 2, single=form == "single")
    assert b.status.item() == 2
    check(bits(b.out)[c:], ref[c:], mag[c:], dot[c:], 900, d)
    # the first sequence over a copy whose block holds zeros
    b.k[b.tables[0, e]] = b.v[b.tables[0, e]] = 0
    ref, mag, dot = b.expect(sees)
    check(bits(b.out)[:c], ref[:c], mag[:c], dot[:c], 900, d)


@pytest.mark.parametrize("window,sinks", [(LARGEST, 0), (LARGEST, LARGEST), (LARGEST - 1, 5), (1, LARGEST)])
@pytest.mark.parametrize("d", [64, 128])
def test_largest_windows_of_chunks_longer_than_their_sequence(d, window, sinks):
    """Rows that stand before the first token, further from it than the window's type has room for."""
    lens, chunks = [10, 0, 130, 64], [300, 40, 500, 65]
    b = Batch(lens, chunks, 4, 2, d, 16, seed=52).upload()
    b.window(window, sinks)
    sees = [np.zeros((c, L), bool) for c, L in zip(chunks, lens)]
    for s, c, L in zip(sees, chunks, lens):
        s[c - min(c, L):] = OS.window_sees(L, min(c, L), window, sinks)
    b.check(sees)
    assert not bits(b.out)[:290].any() and not bits(b.out)[300:340].any()
