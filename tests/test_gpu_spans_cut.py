"""Windowed and tree attention where a run's keys are divided between CTAs or warps and joined again: what is not
a number has to survive the join, whatever the schedule cut.  Bounds and oracle as in test_gpu_spans."""
import numpy as np
import pytest
import torch

from oracle import quant as OQ
from test_gpu_spans import Batch, bits, built, check, tree_words  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

NAN, INF, NINF = 0x7FC0, 0x7F80, 0xFF80


def put(b, x, i, t, value, col=0):
    """Token t of sequence i: `value` in one column, all KV heads."""
    x[b.tables[i][t // b.bs], :, t % b.bs, col] = value


# ------------------------------------------------------------ what is not a number
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 1), (128, 16, 2), (64, 8, 2), (128, 3, 3)])
def test_nan_and_infinite_queries_of_cut_trees(d, Hq, Hkv):
    chunks = [64, 7, 26]
    b = Batch([20000, 5000, 9000], chunks, Hq, Hkv, d, 32, seed=31)
    for row, head, value in ((0, 0, NAN), (5, Hq - 1, INF), (63, 1, NINF), (64, 0, NAN), (70, 2, INF), (96, Hq - 1, NAN)):
        b.q[row, head, (7 * row) % d] = value
    words = tree_words(chunks, b.rng)
    b.upload().tree(words)
    b.check(b.sees_tree(words))


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 4, 1), (64, 4, 2)])
def test_nan_and_infinite_queries_of_cut_windows(d, Hq, Hkv):
    b = Batch([9000, 700, 5000], [100, 3, 300], Hq, Hkv, d, 16, seed=32)
    for row, head, value in ((0, 0, NAN), (60, Hq - 1, INF), (99, 1, NINF), (101, 2, NAN), (103, 0, INF), (402, Hq - 1, NAN)):
        b.q[row, head, (5 * row) % d] = value
    b.upload().window(4000, 4)
    b.check(b.sees_window(4000, 4))


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 1), (64, 32, 2)])
def test_nan_and_infinite_queries_of_single_tokens(d, Hq, Hkv):
    b = Batch([20000, 3, 9000, 700, 40], [1] * 5, Hq, Hkv, d, 16, seed=33)
    for row, head, value in ((0, 0, NAN), (1, 1, INF), (2, Hq - 1, NINF), (3, 2, NAN), (4, 3, NAN)):
        b.q[row, head, (11 * row) % d] = value
    b.upload().window(15000, 4, single=True)
    b.check(b.sees_window(15000, 4))


@pytest.mark.parametrize("window", [1000, 1500, 2000])
def test_a_nan_key_that_is_all_a_piece_shows(window):
    """One sink that every row sees, NaN: the late rows of a query tile see nothing else of the tiles before their
    window, which are a piece of their own where a border falls right behind them."""
    b = Batch([3000], [1024], 8, 8, 128, 16, seed=34)
    put(b, b.k, 0, 0, NAN)
    b.upload().window(window, 1)
    b.check(b.sees_window(window, 1))


@pytest.mark.parametrize("form", ["tree", "chunk", "single"])
@pytest.mark.parametrize("what", ["keys", "values"])
def test_what_is_not_finite_far_below_the_maximum(form, what):
    """One key's score lies 300 log2 units above the others: the other pieces' factors underflow, and what they hold
    shows all the same (an infinite value under an underflowed weight: as an infinity or as NaN)."""
    c = 1 if form == "single" else 5
    b = Batch([20000, 8000], [c, c], 4, 2, 128, 16, seed=35)
    b.q[..., 0] = 0x4220  # 40
    for i, (top, at) in enumerate(((15000, 3000), (900, 7000))):
        put(b, b.k, i, top, 0x4280)  # 64: a score of 226 where others stay below 25
        put(b, b.k if what == "keys" else b.v, i, at, NAN if what == "keys" else INF, 9)
    b.upload()
    words = [1] * (2 * c)
    if form == "tree":
        b.tree(words)
    else:
        b.window(1 << 20, 0, single=form == "single")
    got = OQ.bf16_values(bits(b.out))
    if what == "keys":
        assert np.isnan(got).all()
    else:
        assert not np.isfinite(got[..., 9]).any()
        assert np.isfinite(np.delete(got, 9, -1)).all()
    assert b.status.item() == 0


def test_rows_of_infinitely_low_scores_stay_zeros():
    """Every visible score -inf: zeros, in runs that are cut as in others; the rows beside them are as ever."""
    chunks = [9, 4]
    b = Batch([12000, 300], chunks, 4, 2, 128, 16, seed=36)
    b.k[..., 3] = np.where(b.k[..., 3] == NAN, NAN, 0x3F80)  # 1 in every cached token
    for row, head in ((0, 0), (8, 3), (10, 1)):
        b.q[row, head, 3] = NINF
    zero = np.zeros((13, 4), bool)
    zero[[0, 8, 10], [0, 3, 1]] = True
    words = [1] * 13
    for call, sees in ((lambda: b.tree(words), b.sees_tree(words)), (lambda: b.window(11000, 0), b.sees_window(11000, 0))):
        b.upload()
        call()
        got = bits(b.out)
        ref, mag, dot = b.expect(sees)
        assert not got[zero].any() and not ref[zero].any()
        check(got[~zero], ref[~zero], mag[~zero], dot[~zero], 12000, 128)
        assert b.status.item() == 0
