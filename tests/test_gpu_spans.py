"""Windowed and tree attention on the GPU against the float64 oracle.

Bound.  With s the scores, p the weights, A = max_t scale sum_i |q_i k_ti| over the
keys a row sees, mag = sum_t p_t |v_t| (per output value), n keys:
  * scores: bf16 products are exact in fp32; d of them are summed in fp32, each
    addition off by at most 2^-23 of a partial sum <= A, and a few roundings of the
    scaling: (d + 16) 2^-23 A; every weight is off by that relatively, and so is the
    sum of the weights: twice;
  * 2^x of the hardware, the merges' factors and the final division: 2^-18;
  * fp32 sums over n keys, of weights and of products: 2 n 2^-24;
  * weights are rounded to bf16 for their product with the values: 2^-8 of each;
  * the output's rounding to bf16: 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import quant as OQ
from oracle import rope as OR
from oracle import spans as OS
from paged_kv_cache_276_gb300 import inputs, native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_276_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def gpu_bf16(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(torch.bfloat16)


def dev(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda").to(dtype)


def random_bits(shape, rng, size=1.0):
    return bits(torch.from_numpy(rng.standard_normal(shape) * size).to(torch.bfloat16)).copy()


def check(got, ref, mag, dot, n, d):
    """got [rows, Hq, d] bf16 bits."""
    g = OQ.bf16_values(got)
    rel = 2 * (d + 16) * 2.0 ** -23 * dot[..., None] + 2.0 ** -18 + 2 * n * 2.0 ** -24
    bound = (2.0 ** -8 * (np.abs(ref) + mag) + rel * 2 * mag) * (1 + 2.0 ** -7) + 2.0 ** -130
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(g), nan), "NaN where the oracle has none, or the reverse"
    inf = np.isinf(ref)
    assert np.array_equal(g[inf], ref[inf])
    ok = nan | inf
    err = np.abs(g - np.where(ok, 0.0, ref))[~ok]
    worst = (err / bound[~ok]).max() if err.size else 0.0
    assert worst <= 1.0, f"off by {worst:.3g} times the bound"


class Batch:
    """Sequences of given lengths and chunks over a permuted pool whose unused slots hold `fill`."""

    def __init__(self, lens, chunks, Hq, Hkv, d, bs, seed=0, fill=0x7FC0, spare=3, max_blocks=None):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.bs = [int(x) for x in lens], Hq, Hkv, d, bs
        self.start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        self.NB = sum(-(-n // bs) for n in self.lens) + spare
        self.tables, _ = inputs.permuted_tables(self.lens, bs, self.NB, rng, max_blocks)
        self.k, self.v = (np.full((self.NB, Hkv, bs, d), fill, np.uint16) for _ in "kv")
        for i, L in enumerate(self.lens):
            t = np.arange(L)
            at = self.tables[i][t // bs]
            self.k[at, :, t % bs] = random_bits((L, Hkv, d), rng)
            self.v[at, :, t % bs] = random_bits((L, Hkv, d), rng)
        self.q = random_bits((int(self.start[-1]), Hq, d), rng)
        self.scale = float(np.float32(d ** -0.5))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_len = max(self.lens, default=0)

    def chunk(self, i):
        return int(self.start[i + 1] - self.start[i])

    def upload(self):
        self.gq, self.gk, self.gv = gpu_bf16(self.q), gpu_bf16(self.k), gpu_bf16(self.v)
        self.gt, self.gl = dev(self.tables, torch.int32), dev(np.array(self.lens, np.int64), torch.int32)
        self.gs = dev(self.start, torch.int32)
        self.out = torch.full_like(self.gq, 7.0)
        return self

    def expect(self, sees):
        return OS.attend(self.q, self.k, self.v, self.tables, self.lens, self.start, self.scale, sees)

    def window(self, window, sinks, single=False, workspace="garbage", max_len=None, stream=None):
        n = native.paged_attention_window_workspace_size(len(self.lens), len(self.q), self.Hq, self.Hkv, self.d,
                                                         self.max_len if max_len is None else max_len, window, sinks)
        if workspace == "garbage":
            workspace = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        native.paged_attention_window(self.gq, self.gk, self.gv, self.gt, self.gl,
                                      self.max_len if max_len is None else max_len, window, sinks, self.scale, self.out,
                                      None if single else self.gs, workspace, self.status, stream)
        return self.out

    def tree(self, words, nodes=64, workspace="garbage", max_len=None, stream=None):
        n = native.paged_attention_tree_workspace_size(len(self.lens), len(self.q), nodes, self.Hq, self.Hkv, self.d,
                                                       self.max_len if max_len is None else max_len)
        if workspace == "garbage":
            workspace = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        self.gm = torch.from_numpy(np.asarray(words, dtype=np.uint64).view(np.int64)).cuda()
        native.paged_attention_tree(self.gq, self.gk, self.gv, self.gt, self.gl, self.gs, self.gm, nodes,
                                    self.max_len if max_len is None else max_len, self.scale, self.out, workspace,
                                    self.status, stream)
        return self.out

    def sees_window(self, window, sinks):
        return [OS.window_sees(L, self.chunk(i), window, sinks) for i, L in enumerate(self.lens)]

    def sees_tree(self, words):
        return [OS.tree_sees(L, self.chunk(i), words[self.start[i]:self.start[i + 1]]) for i, L in enumerate(self.lens)]

    def check(self, sees):
        ref, mag, dot = self.expect(sees)
        check(bits(self.out), ref, mag, dot, max([s.sum(-1).max(initial=0) for s in sees], default=0), self.d)
        assert self.status.item() == 0


def tree_words(chunks, rng, density=None):
    """Random trees (ancestors and the node itself), or masks of independent bits."""
    out = []
    for c in chunks:
        m = []
        for j in range(c):
            if density is None:
                parent = int(rng.integers(-1, j)) if j else -1
                m.append((m[parent] if parent >= 0 else 0) | (1 << j))
            else:
                m.append(sum(1 << x for x in range(64) if rng.random() < density))  # bits past the tree too
        out += m
    return out


ODD_LENS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 383, 385, 640, 1001]


# ---------------------------------------------------------- window, single tokens
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (16, 4), (17, 3), (64, 0), (100, 1), (128, 130), (200, 16),
                                          (333, 64), (1001, 0), (5000, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64)])
def test_window_single_tokens(d, bs, window, sinks):
    b = Batch(ODD_LENS + [0], [1] * (len(ODD_LENS) + 1), 4, 2, d, bs, seed=window + sinks + d).upload()
    b.window(window, sinks, single=True)
    b.check(b.sees_window(window, sinks))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (8, 1), (9, 1), (12, 1), (16, 1), (14, 2), (16, 16), (32, 2), (24, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_window_single_tokens_head_layouts(Hq, Hkv, d):
    b = Batch([1, 77, 500, 33, 1030], [1] * 5, Hq, Hkv, d, 16, seed=Hq).upload()
    b.window(300, 5, single=True)
    b.check(b.sees_window(300, 5))


def test_window_single_tokens_many_sequences():
    lens = np.random.default_rng(3).integers(0, 90, 3000).tolist()
    b = Batch(lens, [1] * 3000, 2, 1, 64, 16, seed=4).upload()
    b.window(40, 2, single=True)
    b.check(b.sees_window(40, 2))


@pytest.mark.parametrize("lens,Hq,Hkv,window,sinks", [([30000], 8, 1, 20000, 4), ([9000, 1, 20000, 700], 16, 2, 8192, 0),
                                                      ([40000, 39999], 2, 2, 1 << 20, 0)])
def test_window_single_tokens_long(lens, Hq, Hkv, window, sinks):
    b = Batch(lens, [1] * len(lens), Hq, Hkv, 128, 32, seed=5).upload()
    b.window(window, sinks, single=True)
    b.check(b.sees_window(window, sinks))


# ------------------------------------------------------------------ window, chunks
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 1), (33, 4), (64, 0), (128, 130), (129, 7), (500, 16), (4000, 0)])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64)])
def test_window_chunks(d, bs, window, sinks):
    lens = [1, 5, 64, 300, 257, 700, 129, 1000, 40]
    chunks = [1, 5, 30, 257, 1, 65, 129, 0, 40]
    b = Batch(lens, chunks, 8, 2, d, bs, seed=window + d).upload()
    b.window(window, sinks)
    b.check(b.sees_window(window, sinks))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 1), (7, 1), (8, 1), (11, 1), (16, 1), (6, 2), (16, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_window_chunks_head_layouts(Hq, Hkv, d):
    b = Batch([260, 31, 515], [200, 31, 40], Hq, Hkv, d, 16, seed=Hq + d).upload()
    b.window(100, 3)
    b.check(b.sees_window(100, 3))


def test_window_chunks_longer_than_their_sequence():
    """Rows before the sequence's first token see nothing."""
    b = Batch([10, 0, 5, 130], [25, 7, 5, 200], 4, 2, 64, 16, seed=1).upload()
    b.window(8, 2)
    sees = [np.zeros((b.chunk(i), L), bool) for i, L in enumerate(b.lens)]
    for i, L in enumerate(b.lens):
        full = OS.window_sees(L, min(L, b.chunk(i)), 8, 2)
        sees[i][b.chunk(i) - len(full):] = full
    b.check(sees)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 4, 4)])
def test_a_window_over_everything_is_the_prefill(d, Hq, Hkv):
    b = Batch([900, 33, 300], [600, 33, 1], Hq, Hkv, d, 16, seed=2).upload()
    b.window(900, 0)
    b.check(b.sees_window(900, 0))
    ref = torch.empty_like(b.out)
    native.paged_attention_prefill(b.gq, b.gk, b.gv, b.gt, b.gl, b.gs, b.scale, ref)
    # both are within the bound of the oracle; they round the same weights: a few last places apart
    assert (b.out.float() - ref.float()).abs().max().item() <= 2.0 ** -6 * ref.abs().max().item()


def test_window_long_prompt():
    b = Batch([3000], [2500], 4, 1, 128, 16, seed=8).upload()
    b.window(700, 4)
    b.check(b.sees_window(700, 4))


@pytest.mark.parametrize("window,sinks", [(1, 2 ** 31 - 1), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (50, 2 ** 31 - 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_window_chunks_largest_windows_and_sinks(d, window, sinks):
    b = Batch([700, 64, 1], [300, 64, 1], 8, 2, d, 16, seed=3 + d).upload()
    b.window(window, sinks)
    b.check(b.sees_window(window, sinks))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("longest,window", [(3, 40), (90, 200)])
def test_window_chunks_many_sequences(d, longest, window):
    """More sequences than two CTAs of an SM have room for."""
    rng = np.random.default_rng(11)
    chunks = rng.integers(0, longest + 1, 700)
    lens = chunks + rng.integers(0, 120, 700)
    b = Batch(lens, chunks, 4, 1, d, 16, seed=12).upload()
    b.window(window, 3)
    b.check(b.sees_window(window, 3))


@pytest.mark.parametrize("d,chunk", [(64, 600), (128, 600), (64, 16), (128, 16)])
def test_window_chunks_many_runs(d, chunk):
    """Several runs per CTA, of tiles of 8 tokens, with and without ones that are cut."""
    lens = [700, 640, 600, 655]
    b = Batch(lens, [chunk] * 4, 64, 4, d, 32, seed=13).upload()
    for window, sinks in ((90, 5), (640, 0)):
        b.window(window, sinks)
        b.check(b.sees_window(window, sinks))


@pytest.mark.parametrize("single", [False, True])
def test_blocks_in_several_tables_and_twice_in_one(single):
    """Shared prefixes, and a block that stands at two places of one sequence."""
    b = Batch([200, 200, 333], [1] * 3 if single else [40, 7, 90], 8, 2, 128, 16, seed=14)
    b.tables[1][:10] = b.tables[0][:10]
    b.tables[2][5] = b.tables[2][3]
    b.upload()
    b.window(150, 4, single=single)
    b.check(b.sees_window(150, 4))
    if not single:
        return
    words = tree_words([1] * 3, b.rng)
    b.tree(words)
    b.check(b.sees_tree(words))


# ----------------------------------------------------------------------- trees
@pytest.mark.parametrize("nodes", [1, 2, 7, 8, 26, 33, 63, 64])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 128)])
def test_tree_sizes(d, bs, nodes):
    rng = np.random.default_rng(nodes)
    lens = [nodes, nodes + 1, nodes + 127, nodes + 128, nodes + 200, 513 + nodes, 130, 999]
    chunks = [nodes, nodes, nodes, nodes, max(1, nodes // 2), nodes, 0, 1]
    b = Batch(lens, chunks, 8, 2, d, bs, seed=nodes + d).upload()
    words = tree_words(chunks, rng)
    b.tree(words, nodes)
    b.check(b.sees_tree(words))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 1), (8, 1), (9, 1), (12, 1), (16, 1), (14, 2), (16, 16), (48, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_head_layouts(Hq, Hkv, d):
    rng = np.random.default_rng(Hq)
    chunks = [13, 64, 1, 30]
    b = Batch([200, 700, 90, 31], chunks, Hq, Hkv, d, 16, seed=Hq).upload()
    words = tree_words(chunks, rng)
    b.tree(words)
    b.check(b.sees_tree(words))


@pytest.mark.parametrize("density", [0.0, 0.1, 0.5, 1.0])
def test_tree_any_mask_and_rows_that_see_nothing(density):
    """Masks of independent bits, some past the tree; without a context a zero mask leaves a row empty."""
    rng = np.random.default_rng(6)
    chunks = [20, 64, 33, 1, 64, 5]
    b = Batch([20, 64, 33 + 95, 1, 64 + 300, 5], chunks, 6, 2, 64, 16, seed=6).upload()
    words = tree_words(chunks, rng, density)
    b.tree(words)
    b.check(b.sees_tree(words))


def test_tree_with_fewer_tokens_than_nodes():
    """Nodes before the sequence's start do not exist: their bits count for nothing."""
    chunks = [10, 3, 6]
    b = Batch([4, 0, 6], chunks, 4, 2, 64, 16, seed=7).upload()
    words = [(1 << 64) - 1] * 19
    b.tree(words, 16)
    sees = [np.ones((10, 4), bool), np.zeros((3, 0), bool), np.ones((6, 6), bool)]
    b.check(sees)


@pytest.mark.parametrize("lens,chunks,Hq,Hkv", [([30000], [64], 8, 1), ([9000, 70, 20000, 700], [26, 8, 64, 33], 16, 2),
                                                ([20000], [5], 2, 2), ([16384, 16384, 16384], [64, 64, 64], 16, 1)])
def test_tree_long_contexts(lens, chunks, Hq, Hkv):
    rng = np.random.default_rng(9)
    b = Batch(lens, chunks, Hq, Hkv, 128, 32, seed=9).upload()
    words = tree_words(chunks, rng)
    b.tree(words)
    b.check(b.sees_tree(words))


def test_tree_many_sequences():
    rng = np.random.default_rng(10)
    chunks = rng.integers(0, 9, 1024)
    lens = chunks + rng.integers(0, 60, 1024)
    b = Batch(lens, chunks, 2, 1, 64, 16, seed=10).upload()
    words = tree_words(chunks, rng)
    b.tree(words, 8)
    b.check(b.sees_tree(words))


def test_a_chain_is_causal_attention():
    """A tree without branches is a causal chunk: the window's answer with a window over everything."""
    b = Batch([300, 20, 1500], [9, 20, 64], 8, 2, 128, 16, seed=11).upload()
    words = [(1 << (r + 1)) - 1 for c in (9, 20, 64) for r in range(c)]
    b.tree(words)
    b.check(b.sees_window(2000, 0))


# --------------------------------------------- what a row does not see never shows
AWKWARD = np.array([0x7FC0, 0x7F80, 0xFF80, 0x7F7F, 0xFF7F], np.uint16)  # NaN, infinities, the type's largest


@pytest.mark.parametrize("d,bs,window,sinks", [(128, 16, 50, 3), (64, 64, 130, 0), (128, 128, 70, 130), (64, 16, 1, 1)])
def test_hidden_tokens_of_single_rows_never_show(d, bs, window, sinks):
    lens = [1, 40, 129, 500, 300, 1000]
    b = Batch(lens, [1] * 6, 4, 2, d, bs, seed=12)
    sees = b.sees_window(window, sinks)
    for i, L in enumerate(lens):
        t = np.nonzero(~sees[i].any(0))[0]
        at = b.tables[i][t // bs]
        for x in (b.k, b.v):
            x[at, :, t % bs] = b.rng.choice(AWKWARD, (len(t), b.Hkv, d))
    b.upload().window(window, sinks, single=True)
    b.check(sees)


@pytest.mark.parametrize("d,bs", [(128, 16), (64, 64), (128, 128)])
@pytest.mark.parametrize("what", ["keys", "values"])
def test_awkward_tokens_show_only_where_they_are_seen(d, bs, what):
    """A chunk's own tokens among them: rows that see one show it, the others do not."""
    lens, chunks = [400, 129, 700, 64], [300, 129, 200, 64]
    b = Batch(lens, chunks, 4, 2, d, bs, seed=13)
    for i, L in enumerate(lens):
        t = b.rng.choice(L, max(1, L // 60), replace=False)
        x = (b.k if what == "keys" else b.v)
        for y in t:
            x[b.tables[i][y // bs], :, y % bs, b.rng.integers(0, d, 3)] = b.rng.choice(AWKWARD[:3])
    b.upload().window(60, 5)
    b.check(b.sees_window(60, 5))


@pytest.mark.parametrize("d,bs,Hq", [(128, 16, 8), (64, 64, 2), (128, 128, 16)])
@pytest.mark.parametrize("what", ["keys", "values"])
def test_awkward_siblings_never_show(d, bs, Hq, what):
    rng = np.random.default_rng(14)
    chunks = [26, 64, 8, 40]
    lens = [26 + 100, 64, 8 + 500, 40 + 128]
    b = Batch(lens, chunks, Hq, 2, d, bs, seed=14)
    words = tree_words(chunks, rng)
    for i, L in enumerate(lens):
        for j in rng.choice(chunks[i], 3, replace=False):  # nodes that few others descend from
            t = L - chunks[i] + int(j)
            (b.k if what == "keys" else b.v)[b.tables[i][t // bs], :, t % bs, rng.integers(0, d, 2)] = \
                rng.choice(AWKWARD[:3])
    b.upload().tree(words)
    b.check(b.sees_tree(words))


def test_blocks_that_were_given_back_are_not_read():
    """Table entries between the sinks and the window may hold anything: no status, the same answer."""
    for single in (True, False):
        lens = [700, 90, 1300, 257]
        chunks = [1] * 4 if single else [100, 90, 33, 1]
        b = Batch(lens, chunks, 4, 2, 128, 16, seed=15)
        window, sinks = 130, 20
        sees = b.sees_window(window, sinks)
        ref, mag, dot = b.expect(sees)
        for i, L in enumerate(lens):
            for e in range(-(-L // 16)):
                if not sees[i][:, e * 16:(e + 1) * 16].any():
                    b.tables[i][e] = [-1, 1 << 30, -(1 << 31), b.NB][e % 4]
        b.upload().window(window, sinks, single=single)
        check(bits(b.out), ref, mag, dot, 150, 128)
        assert b.status.item() == 0


def test_infinite_and_nan_queries_stay_in_their_row():
    b = Batch([100, 300], [40, 64], 4, 2, 128, 16, seed=16)
    b.q[5, 1, 7], b.q[50, 0, 0], b.q[103, 3, 127] = 0x7F80, 0x7FC0, 0xFF80
    b.upload().window(90, 2)
    got = OQ.bf16_values(bits(b.out))
    ref, mag, dot = b.expect(b.sees_window(90, 2))
    bad = np.zeros((104, 4), bool)
    bad[5, 1] = bad[50, 0] = bad[103, 3] = True
    assert np.isnan(got[bad]).all(-1).all() or not np.isfinite(got[bad]).all()
    check(bits(b.out)[~bad], ref[~bad], mag[~bad], dot[~bad], 92, 128)


@pytest.mark.parametrize("scale", [0.0, -0.4, 30.0, 1e-30])
def test_scales(scale):
    b = Batch([200, 77], [64, 20], 4, 2, 64, 16, seed=17)
    b.scale = float(np.float32(scale))
    b.upload().window(50, 3)
    b.check(b.sees_window(50, 3))
    words = tree_words([64, 20], np.random.default_rng(1))
    b.tree(words)
    b.check(b.sees_tree(words))
    b1 = Batch([200, 77], [1, 1], 4, 2, 64, 16, seed=17)
    b1.scale = b.scale
    b1.upload().window(50, 3, single=True)
    b1.check(b1.sees_window(50, 3))


# ------------------------------------------------------------- bad device arguments
def test_bad_lengths_blocks_and_starts_are_reported():
    def fresh(chunks=(4, 4, 4)):
        return Batch([60, 90, 40], list(chunks), 4, 2, 64, 16, seed=18)

    words = [15] * 12
    for call in (lambda b: b.window(30, 2), lambda b: b.tree(words, 4)):
        b = fresh().upload()
        b.gl[1] = -3
        call(b)
        assert b.status.item() == 4
        assert not bits(b.out)[4:8].any()  # no keys: zeros
        b = fresh().upload()
        b.gl[2] = 10 ** 6  # clamped to max_seq_len or the table
        call(b)
        assert b.status.item() & 4
        for bad in (-1, 10 ** 6, 1 << 31 - 1):
            b = fresh().upload()
            b.gt[0, 3] = min(bad, 2 ** 31 - 1)
            call(b)
            assert b.status.item() == 2
            ref, mag, dot = b.expect(b.sees_window(30, 2) if call.__code__.co_consts and "window" in call.__code__.co_names
                                     else b.sees_tree(words))
            check(bits(b.out)[4:], ref[4:], mag[4:], dot[4:], 90, 64)
        for at, val in ((1, 100), (2, -1), (1, 9)):
            b = fresh().upload()
            b.gs[at] = val
            call(b)
            assert b.status.item() & 16
    b = fresh((4, 6, 2)).upload()  # a tree of more nodes than the bound
    b.tree(words, 4)
    assert b.status.item() == 16
    assert (bits(b.out)[4:10] == bits(torch.tensor([7.0], dtype=torch.bfloat16))[0]).all()
    for single in (True,):
        b = Batch([60, 90, 40], [1] * 3, 4, 2, 64, 16, seed=18).upload()
        b.gl[1] = -3
        b.gt[2, 2] = b.NB
        b.window(30, 2, single=True)
        assert b.status.item() == 4 | 2
        assert not bits(b.out)[1].any()


def test_rows_of_no_sequence_stay():
    b = Batch([60, 90], [5, 7], 4, 2, 64, 16, seed=19)
    b.q = np.concatenate([b.q, b.q[:9]])
    b.upload()
    b.window(30, 2)
    assert (b.out[12:] == 7.0).all() and not (b.out[:12] == 7.0).all(-1).any()
    b.out.fill_(7.0)
    b.tree([1] * 21, 8)
    assert (b.out[12:] == 7.0).all() and not (b.out[:12] == 7.0).all(-1).any()


def test_lengths_above_the_bound_are_clamped():
    b = Batch([500, 300], [1, 1], 4, 2, 64, 16, seed=20).upload()
    b.window(60, 2, single=True, max_len=400)
    assert b.status.item() == 4
    b.lens[0] = 400
    ref, mag, dot = b.expect(b.sees_window(60, 2))
    check(bits(b.out), ref, mag, dot, 64, 64)


# ------------------------------------------------------ streams, graphs, workspaces
def mixed_cases():
    """(name, call(batch, workspace, stream), workspace bytes) over one batch of uneven lengths."""
    single = Batch([5000, 40, 900, 2500], [1] * 4, 16, 2, 128, 16, seed=21)
    chunk = Batch([1200, 40, 900, 2500], [300, 40, 7, 129], 8, 2, 128, 16, seed=22)
    tree = Batch([3000, 40, 900, 7000], [26, 40, 7, 64], 8, 2, 128, 16, seed=23)
    words = tree_words([26, 40, 7, 64], np.random.default_rng(3))
    return [("single", single, lambda ws, st=None: single.window(3000, 4, True, ws, stream=st), single.sees_window(3000, 4)),
            ("chunk", chunk, lambda ws, st=None: chunk.window(500, 4, False, ws, stream=st), chunk.sees_window(500, 4)),
            ("tree", tree, lambda ws, st=None: tree.tree(words, 64, ws, stream=st), tree.sees_tree(words))]


def size_of(name, b):
    if name == "tree":
        return native.paged_attention_tree_workspace_size(4, len(b.q), 64, b.Hq, b.Hkv, b.d, b.max_len)
    w = (3000, 4) if name == "single" else (500, 4)
    return native.paged_attention_window_workspace_size(4, len(b.q), b.Hq, b.Hkv, b.d, b.max_len, *w)


def test_repeats_bit_for_bit():
    for name, b, call, sees in mixed_cases():
        b.upload()
        call("garbage")
        first = bits(b.out)
        b.check(sees)
        for _ in range(5):
            call("garbage")
            assert np.array_equal(bits(b.out), first), name


def test_captured_calls_share_a_workspace_and_follow_their_inputs():
    cases = mixed_cases()
    ws = torch.full((max(16, max(size_of(n, b) for n, b, _, _ in cases)),), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    for name, b, call, sees in cases:
        b.upload()
        call(ws)
        torch.cuda.synchronize()
        if name == "tree":
            words = b.gm.clone()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                native.paged_attention_tree(b.gq, b.gk, b.gv, b.gt, b.gl, b.gs, words, 64, b.max_len, b.scale, b.out, ws,
                                            b.status)
            b.keep = words
        else:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(ws)
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for _, b, _, sees in cases:
        b.check(sees)
    # shorter sequences and other queries, the same graphs
    for name, b, _, _ in cases:
        b.lens = [max(b.chunk(i), L // 3) for i, L in enumerate(b.lens)]
        b.gl.copy_(dev(np.array(b.lens), torch.int32))
        b.q = random_bits(b.q.shape, b.rng)
        b.gq.copy_(gpu_bf16(b.q))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for name, b, _, _ in cases:
        if name == "single":
            b.check(b.sees_window(3000, 4))
        elif name == "chunk":
            b.check(b.sees_window(500, 4))
        else:
            b.check(b.sees_tree(b.keep.cpu().numpy().view(np.uint64).tolist()))


def test_two_streams_at_once_with_a_workspace_each():
    cases = mixed_cases()
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [torch.full((max(16, size_of(n, b)),), 0xFF, dtype=torch.uint8, device="cuda") for n, b, _, _ in cases]
    for _, b, _, _ in cases:
        b.upload()
    torch.cuda.synchronize()
    for _ in range(4):
        for (_, _, call, _), s, ws in zip(cases, streams, spaces):
            call(ws, s)
    torch.cuda.synchronize()
    for _, b, _, sees in cases:
        b.check(sees)


def test_back_to_back_calls_over_one_workspace():
    cases = mixed_cases()
    ws = torch.full((max(16, max(size_of(n, b) for n, b, _, _ in cases)),), 0xFF, dtype=torch.uint8, device="cuda")
    for _, b, _, _ in cases:
        b.upload()
    for _ in range(3):
        for _, b, call, _ in cases:
            call(ws)
    for _, b, _, sees in cases:
        b.check(sees)


def test_offsets_past_32_bits():
    """Blocks beyond 4 GiB of the cache."""
    Hkv, bs, d = 8, 128, 128
    NB = (1 << 33) // (Hkv * bs * d * 2) + 5
    b = Batch([500, 129], [64, 30], 8, Hkv, d, bs, seed=24)
    far = NB - b.NB
    k = torch.zeros((NB, Hkv, bs, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[far:], v[far:] = gpu_bf16(b.k), gpu_bf16(b.v)
    b.upload()
    b.gk, b.gv, b.gt = k, v, torch.where(b.gt >= 0, b.gt + far, b.gt)
    b.window(200, 4)
    b.check(b.sees_window(200, 4))
    words = tree_words([64, 30], b.rng)
    b.tree(words)
    b.check(b.sees_tree(words))
    one = Batch([500, 129], [1, 1], 8, Hkv, d, bs, seed=24).upload()
    one.gk, one.gv, one.gt = k, v, torch.where(one.gt >= 0, one.gt + far, one.gt)
    k[far:], v[far:] = gpu_bf16(one.k), gpu_bf16(one.v)
    one.window(200, 4, single=True)
    one.check(one.sees_window(200, 4))


# ------------------------------------------------------------ a run of them together
def test_a_drafted_step_of_a_rotary_model():
    """Two layers, one over the whole context, one windowed: a prompt is appended and attended, a tree is drafted
    on a copy-on-write fork and verified, its accepted path is appended to the sequence itself, and the next
    token is decoded over it.  Every attention against the oracle over a host copy of the cache."""
    rng = np.random.default_rng(25)
    Hq, Hkv, d, bs, NB, rot = 8, 2, 128, 16, 40, 128
    scale = float(np.float32(d ** -0.5))
    cs = OR.table(400, rot)
    table = torch.from_numpy(cs).cuda()
    alloc = native.BlockAllocator(NB, bs)
    caches = [[torch.zeros((NB, Hkv, bs, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"] for _ in range(2)]
    window, sinks = 70, 4
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, native.paged_attention_tree_workspace_size(1, 300, 64, Hq, Hkv, d, 400),
                         native.paged_attention_window_workspace_size(1, 300, Hq, Hkv, d, 400, window, sinks)),
                     dtype=torch.uint8, device="cuda")

    def append(layer, seq_slots, positions, qkv):
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
        native.pkv_write_rope(q, k, v, dev(positions, torch.int64), table, dev(seq_slots, torch.int64), out,
                              *caches[layer], d_status=st)
        return out

    def tables_of(seq):
        t, lens = alloc.block_table([seq], 25)
        return np.asarray(t, dtype=np.int32), np.asarray(lens, dtype=np.int32)

    def verify(layer, q, out, seq, sees):
        t, lens = tables_of(seq)
        ref, mag, dot = OS.attend(bits(q), *[bits(c) for c in caches[layer]], t, lens, [0, len(q)], scale, [sees])
        check(bits(out), ref, mag, dot, int(lens[0]), d)

    def projection(n):
        return gpu_bf16(random_bits((n, Hq + 2 * Hkv, d), rng))

    def windowed(layer, q, seq, single=False):
        t, lens = tables_of(seq)
        out = torch.empty_like(q)
        native.paged_attention_window(q, *caches[layer], dev(t, torch.int32), dev(lens, torch.int32), int(lens[0]),
                                      window if layer else 400, sinks if layer else 0, scale, out,
                                      None if single else dev([0, len(q)], torch.int32), ws, st)
        verify(layer, q, out, seq, OS.window_sees(int(lens[0]), len(q), window if layer else 400, sinks if layer else 0))

    alloc.seq_add(1)
    n = 150
    slots = alloc.seq_append(1, n)
    for layer in range(2):
        windowed(layer, append(layer, slots, np.arange(n), projection(n)), 1)

    # the tree on a fork, so that the sequence keeps its own blocks
    parents = [-1, -1, 0, 0, 1, 2, 2, 3]
    depth, words = [], []
    for j, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        words.append((1 << j) | (words[p] if p >= 0 else 0))
    alloc.seq_fork(1, 2)
    pair = alloc.seq_cow(2)
    assert pair is not None
    for c in caches:
        native.pkv_block_copy(*c, dev(np.array([pair]), torch.int32), st)
    slots = alloc.seq_append(2, len(parents))
    drafts = [projection(len(parents)) for _ in range(2)]
    mask = dev(np.array(words), torch.int64)
    t, lens = tables_of(2)
    for layer in range(2):
        q = append(layer, slots, n + np.array(depth), drafts[layer])
        out = torch.empty_like(q)
        native.paged_attention_tree(q, *caches[layer], dev(t, torch.int32), dev(lens, torch.int32),
                                    dev([0, len(q)], torch.int32), mask, 8, int(lens[0]), scale, out, ws, st)
        verify(layer, q, out, 2, OS.tree_sees(int(lens[0]), len(parents), words))
    alloc.seq_free(2)

    # nodes 0, 2, 6 were accepted: their rows go to the sequence's next slots, the others nowhere
    path = [0, 2, 6]
    slots = np.full(len(parents), -1, np.int64)
    slots[path] = alloc.seq_append(1, len(path))
    for layer in range(2):
        append(layer, slots, n + np.array(depth), drafts[layer])
    slots = alloc.seq_append(1, 1)
    for layer in range(2):
        windowed(layer, append(layer, slots, [n + 3], projection(1)), 1, single=True)
    assert st.item() == 0
    alloc.close()
