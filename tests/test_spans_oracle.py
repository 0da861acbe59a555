"""Host side of the rotary append, windowed and tree attention: the oracles against
plain loops, refusals of the C ABI and of the Python calls (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import quant as OQ
from oracle import rope as OR
from oracle import spans as OS


@pytest.fixture(scope="module")
def native():
    from paged_kv_cache_276_gb300 import build, native
    build.build()
    native.lib()
    return native


# ------------------------------------------------------------------ oracles
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_oracle_against_complex_numbers(interleaved):
    rng = np.random.default_rng(3)
    T, H, d, rot = 5, 2, 32, 16
    cs = OR.table(50, rot)
    pos, x = rng.integers(0, 50, T), rng.standard_normal((T, H, d))
    y = OR.rotate(x, cs, pos, interleaved, np.float64)
    i, j = OR.pairs(rot, interleaved)
    z = (x[..., i] + 1j * x[..., j]) * (cs[pos, :rot // 2] + 1j * cs[pos, rot // 2:].astype(np.float64))[:, None]
    assert np.allclose(y[..., i], z.real, atol=1e-15) and np.allclose(y[..., j], z.imag, atol=1e-15)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    assert np.allclose(cs[7, 3], np.cos(7 * 10000.0 ** (-6 / 16)), atol=1e-7)


def test_bf16_rounding_oracle_against_torch():
    x = np.random.default_rng(0).integers(0, 1 << 32, 4096, dtype=np.uint64).astype(np.uint32).view(np.float32)
    want = torch.from_numpy(x.copy()).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    keep = ~np.isnan(x)
    assert np.array_equal(OR.to_bf16(x)[keep], want[keep])


def test_row_quantiser_agrees_with_the_bf16_one():
    bits = np.random.default_rng(1).integers(0, 1 << 16, (64, 16)).astype(np.uint16)
    for got, want in zip(OR.quantise(OQ.bf16_values(bits)), OQ.quantise(bits)):
        assert np.array_equal(got, want)


def test_attention_oracle_against_a_plain_loop():
    rng = np.random.default_rng(2)
    B, Hkv, G, d, bs, NB, scale = 3, 2, 3, 16, 4, 12, 0.3
    val = lambda *s: np.round(rng.standard_normal(s) * 8) / 8  # noqa: E731
    q, k, v = val(9, Hkv * G, d), val(NB, Hkv, bs, d), val(NB, Hkv, bs, d)
    lens, start = [7, 2, 13], [0, 3, 4, 9]
    tables = np.array([rng.permutation(NB)[:4] for _ in range(B)])
    words = [0b001, 0b011, 0b101, 0, 0b1, 0b11, 0b101, 0b1101, 0b10001]
    for kind in ("window", "tree"):
        sees = [OS.window_sees(L, start[i + 1] - start[i], 3, 1) if kind == "window" else
                OS.tree_sees(L, start[i + 1] - start[i], words[start[i]:start[i + 1]]) for i, L in enumerate(lens)]
        out = OS.attend(OQ.bf16_bits(q), OQ.bf16_bits(k), OQ.bf16_bits(v), tables, lens, start, scale, sees)[0]
        for i, L in enumerate(lens):
            c = start[i + 1] - start[i]
            for r in range(c):
                row, p = start[i] + r, L - c + r
                for g in range(Hkv * G):
                    num, den = np.zeros(d), 0.0
                    for t in range(L):
                        if kind == "window":
                            ok = t <= p and (p - t < 3 or t < 1)
                        else:
                            ok = t < L - c or words[row] & (1 << (t - (L - c)))
                        if ok:
                            at = tables[i][t // bs], g // G, t % bs
                            w = np.exp(scale * q[row, g] @ k[at])
                            num, den = num + w * v[at], den + w
                    assert np.allclose(out[row, g], num / den if den else 0.0, rtol=1e-12)


# ----------------------------------------------------------------- refusals
F = 1 << 20  # an address that no call dereferences: every case fails a check first
ARG, UNSUPPORTED, WORKSPACE = -1, -4, -8


def rope_args(quant, **kw):
    a = dict(q=F, k=F, v=F, qs=1024, ks=256, vs=256, pos=F, cs=F, top=64, rot=128, inter=0, slots=F, T=4, qo=F,
             qos=1024)
    a.update(dict(kc=F, vc=F, ke=F, ve=F) if quant else dict(kc=F, vc=F))
    a.update(NB=8, bs=16, Hq=8, Hkv=2, d=128, st=None, stream=None)
    a.update(kw)
    return list(a.values())


ROPE_BAD = [(dict(T=-1), ARG), (dict(NB=-1), ARG), (dict(bs=0), ARG), (dict(Hkv=0), ARG), (dict(Hq=-1), ARG),
            (dict(d=0), ARG), (dict(d=24), UNSUPPORTED), (dict(d=528), UNSUPPORTED), (dict(rot=0), ARG),
            (dict(rot=144), ARG), (dict(rot=24), UNSUPPORTED), (dict(top=-1), ARG), (dict(inter=2), ARG),
            (dict(qs=1016), ARG), (dict(qs=1028), ARG), (dict(qos=1023), ARG), (dict(ks=248), ARG), (dict(vs=260), ARG),
            (dict(q=None), ARG), (dict(qo=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(pos=None), ARG),
            (dict(cs=None), ARG), (dict(slots=None), ARG), (dict(kc=None), ARG), (dict(vc=None), ARG),
            (dict(q=F + 8), ARG), (dict(qo=F + 2), ARG), (dict(k=F + 8), ARG), (dict(v=F + 4), ARG),
            (dict(cs=F + 4), ARG), (dict(pos=F + 4), ARG), (dict(slots=F + 4), ARG), (dict(kc=F + 8), ARG),
            (dict(vc=F + 1), ARG)]


@pytest.mark.parametrize("kw,rc", ROPE_BAD)
@pytest.mark.parametrize("quant", [False, True])
def test_rope_refuses(native, quant, kw, rc):
    f = native.lib().pkv_write_rope_quant if quant else native.lib().pkv_write_rope
    assert f(*rope_args(quant, **kw)) == rc


def test_rope_refuses_missing_exponents(native):
    for kw in (dict(ke=None), dict(ve=None)):
        assert native.lib().pkv_write_rope_quant(*rope_args(True, **kw)) == ARG


def window_args(**kw):
    a = dict(q=F, kc=F, vc=F, tbl=F, maxb=8, lens=F, qs=F, B=2, n=4, maxlen=64, window=16, sinks=2, Hq=8, Hkv=2, d=128,
             bs=16, NB=8, scale=0.1, out=F, ws=F, wsb=1 << 40, st=None, stream=None)
    a.update(kw)
    return list(a.values())


def tree_args(**kw):
    a = dict(q=F, kc=F, vc=F, tbl=F, maxb=8, lens=F, qs=F, mask=F, B=2, n=4, nodes=8, maxlen=64, Hq=8, Hkv=2, d=128,
             bs=16, NB=8, scale=0.1, out=F, ws=F, wsb=1 << 40, st=None, stream=None)
    a.update(kw)
    return list(a.values())


SPANS_BAD = [(dict(B=-1), ARG), (dict(n=-1), ARG), (dict(maxb=-1), ARG), (dict(maxlen=-1), ARG), (dict(Hq=0), ARG),
             (dict(Hkv=0), ARG), (dict(Hq=7), ARG), (dict(NB=-1), ARG), (dict(NB=0), ARG),
             (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(d=96), UNSUPPORTED),
             (dict(Hq=34), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(bs=48), UNSUPPORTED),
             (dict(B=1025, n=2000), UNSUPPORTED), (dict(maxb=1 << 27), UNSUPPORTED), (dict(NB=1 << 26), UNSUPPORTED),
             (dict(q=None), ARG), (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(tbl=None), ARG),
             (dict(lens=None), ARG), (dict(out=None), ARG), (dict(q=F + 8), ARG), (dict(kc=F + 8), ARG),
             (dict(vc=F + 2), ARG), (dict(out=F + 4), ARG), (dict(tbl=F + 2), ARG), (dict(lens=F + 1), ARG),
             (dict(qs=F + 2), ARG)]


@pytest.mark.parametrize("kw,rc", SPANS_BAD + [
    (dict(window=0), ARG), (dict(window=-5), ARG), (dict(sinks=-1), ARG), (dict(qs=None), ARG),  # 4 rows of 2 sequences
    (dict(qs=None, B=65536, n=65536), UNSUPPORTED)])
def test_window_refuses(native, kw, rc):
    assert native.lib().paged_attention_window(*window_args(**kw)) == rc


@pytest.mark.parametrize("kw,rc", SPANS_BAD + [
    (dict(nodes=0), ARG), (dict(nodes=65), ARG), (dict(qs=None), ARG), (dict(mask=None), ARG), (dict(mask=F + 4), ARG)])
def test_tree_refuses(native, kw, rc):
    assert native.lib().paged_attention_tree(*tree_args(**kw)) == rc


def test_nothing_to_do_is_a_no_op(native):
    for quant in (False, True):
        f = native.lib().pkv_write_rope_quant if quant else native.lib().pkv_write_rope
        assert f(*rope_args(quant, T=0, q=None, k=None, pos=None, kc=None)) == 0
    f, g = native.lib().paged_attention_window, native.lib().paged_attention_tree
    assert f(*window_args(B=0, n=0, q=None, qs=None)) == 0 and f(*window_args(n=0, q=None)) == 0
    assert g(*tree_args(B=0, q=None)) == 0 and g(*tree_args(n=0, q=None, mask=None)) == 0


def test_attention_refuses_a_missing_or_small_workspace(native):
    lib = native.lib()
    size = native.paged_attention_window_workspace_size(2, 4, 8, 2, 128, 100000, 5000, 4)
    kw = dict(maxlen=100000, maxb=10000, window=5000, sinks=4)
    if size:
        for bad in (dict(ws=None, wsb=0), dict(ws=F, wsb=size - 1), dict(ws=F + 8, wsb=size)):
            assert lib.paged_attention_window(*window_args(**kw, **bad)) == WORKSPACE
    size = native.paged_attention_tree_workspace_size(2, 4, 8, 8, 2, 128, 100000)
    kw = dict(maxlen=100000, maxb=10000)
    if size:
        for bad in (dict(ws=None, wsb=0), dict(ws=F, wsb=size - 1), dict(ws=F + 8, wsb=size)):
            assert lib.paged_attention_tree(*tree_args(**kw, **bad)) == WORKSPACE


def test_workspace_size_of_invalid_sizes_is_zero(native):
    f, g = native.paged_attention_window_workspace_size, native.paged_attention_tree_workspace_size
    for bad in (dict(B=-1), dict(n=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(Hq=64), dict(d=96), dict(L=-1),
                dict(w=0), dict(s=-1), dict(B=0), dict(n=0)):
        a = dict(B=2, n=4, Hq=8, Hkv=2, d=128, L=5000, w=100, s=4)
        a.update(bad)
        assert f(*a.values()) == 0, bad
    for bad in (dict(B=-1), dict(n=-1), dict(T=0), dict(T=65), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(Hq=64),
                dict(d=96), dict(L=-1), dict(B=0), dict(n=0)):
        a = dict(B=2, n=4, T=8, Hq=8, Hkv=2, d=128, L=5000)
        a.update(bad)
        assert g(*a.values()) == 0, bad


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_rope_python_checks(native):
    slots, pos = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int64)
    q, kv, cs = bf(3, 4, 64), bf(3, 2, 64), torch.zeros((9, 32))
    kc = [bf(4, 2, 16, 64), bf(4, 2, 16, 64)]
    f8 = [torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in "kv"]
    f8 += [torch.zeros((4, 2, 16), dtype=torch.uint8) for _ in "kv"]
    for f, cache in ((native.pkv_write_rope, kc), (native.pkv_write_rope_quant, f8)):
        with pytest.raises(ValueError, match="CUDA"):
            f(q, kv, kv, pos, cs, slots, q, *cache)
        for args in ((q, kv.float(), kv, pos, cs, slots, q), (q, kv, kv, pos.int(), cs, slots, q),
                     (q, kv, kv, pos, cs.double(), slots, q), (q, kv, kv, pos, cs, [0, 1, 2], q),
                     (q, None, kv, pos, cs, slots, q), (q.float(), kv, kv, pos, cs, slots, q)):
            with pytest.raises(TypeError):
                f(*args, *cache)
        for args in ((q, kv[:2], kv, pos, cs, slots, q), (q, kv, kv, pos[:2], cs, slots, q),
                     (q, kv, kv, pos, cs[0], slots, q), (q, kv, kv, pos, cs, slots, None),
                     (None, kv, kv, pos, cs, slots, q), (q, kv, kv, pos, cs, slots, bf(3, 5, 64)),
                     (q[:, 0], kv, kv, pos, cs, slots, q), (q[:2], kv, kv, pos, cs, slots, q),
                     (q, kv[:1].expand(3, 2, 64), kv, pos, cs, slots, q),
                     (q, bf(3, 64, 2).transpose(1, 2), kv, pos, cs, slots, q)):
            with pytest.raises(ValueError):
                f(*args, *cache)
        with pytest.raises((TypeError, ValueError)):
            f(q, kv, kv, pos, cs, slots, q, *cache[::-1][:-1], bf(4, 2, 8, 64))
        with pytest.raises(TypeError, match="d_status"):
            f(q, kv, kv, pos, cs, slots, q, *cache, d_status=torch.zeros(1))


def test_attention_python_checks(native):
    q, kc = bf(5, 4, 64), bf(4, 2, 16, 64)
    tbl, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    qs, mask = torch.tensor([0, 2, 5], dtype=torch.int32), torch.zeros(5, dtype=torch.int64)

    def window(q=q, kc=kc, vc=kc, tbl=tbl, lens=lens, out=None, qs=qs, ws=None, st=None):
        native.paged_attention_window(q, kc, vc, tbl, lens, 40, 8, 1, 0.1, q.clone() if out is None else out, qs, ws, st)

    def tree(q=q, kc=kc, vc=kc, tbl=tbl, lens=lens, out=None, qs=qs, mask=mask, ws=None, st=None):
        native.paged_attention_tree(q, kc, vc, tbl, lens, qs, mask, 8, 40, 0.1, q.clone() if out is None else out, ws, st)

    for f in (window, tree):
        with pytest.raises(ValueError, match="CUDA"):
            f()
        for kw in (dict(q=q.float(), out=q), dict(kc=kc.float()), dict(tbl=tbl.long()), dict(lens=lens.long()),
                   dict(qs=qs.long()), dict(st=torch.zeros(1)), dict(vc=3)):
            with pytest.raises(TypeError):
                f(**kw)
        for kw in (dict(q=q[0], out=q[0]), dict(out=q[:3]), dict(tbl=tbl[:1]), dict(tbl=tbl[0]), dict(qs=qs[:2]),
                   dict(vc=kc[:2]), dict(q=bf(5, 4, 128)), dict(ws=3), dict(ws=torch.zeros((4, 4)).t()[1:])):
            with pytest.raises(ValueError):
                f(**kw)
    with pytest.raises(ValueError):  # one row per sequence without q_start
        window(qs=None)
    with pytest.raises(TypeError):
        tree(qs=None)
    with pytest.raises(TypeError):
        tree(mask=None)
    with pytest.raises(TypeError):
        tree(mask=mask.int())
    with pytest.raises(ValueError):
        tree(mask=mask[:3])
