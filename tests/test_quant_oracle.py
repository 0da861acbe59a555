"""The 8-bit cache on the CPU: the oracle's pins, and the library's refusals
(argument checks that run on the host before anything is launched)."""
import numpy as np
import pytest
import torch

from oracle import quant as OQ


@pytest.fixture(scope="module")
def native():
    from paged_kv_cache_276_gb300 import build, native
    build.build()
    return native


# ------------------------------------------------------------- the oracle's pins
def test_code_values_match_the_type():
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn)
    got = codes.to(torch.float64).numpy()
    assert np.array_equal(got, OQ.TABLE, equal_nan=True)
    assert np.nanmax(OQ.TABLE) == 448.0 and OQ.TABLE[1] == 2.0 ** -9


def test_encode_inverts_every_code_and_rounds_ties_to_even():
    finite = [c for c in range(256) if not np.isnan(OQ.TABLE[c])]
    assert OQ.encode(OQ.TABLE[finite]).tolist() == finite
    assert OQ.encode(np.array([np.nan]))[0] == 0x7F
    pos = np.sort(OQ.TABLE[:127])
    mid = (pos[1:] + pos[:-1]) / 2  # half way: the even one of the two neighbours
    assert all(c % 2 == 0 for c in OQ.encode(mid).tolist())
    assert np.array_equal(OQ.encode(mid * (1 + 1e-12)), OQ.encode(pos[1:]))
    assert np.array_equal(OQ.encode(mid * (1 - 1e-12)), OQ.encode(pos[:-1]))
    assert OQ.TABLE[OQ.encode(np.array([1e9, -1e9]))].tolist() == [448.0, -448.0]


def test_encode_agrees_with_the_cast():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000)).clip(-448, 448).astype(np.float32)
    cast = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OQ.encode(x.astype(np.float64)), cast)


@pytest.mark.parametrize("top,e", [(448.0, 0), (450.0, 1), (224.0, -1), (226.0, 0), (1.0, -8), (1.75, -8), (1.765625, -7),
                                   (0.0, -31), (2.0 ** -40, -31), (2.0 ** 60, 31)])
def test_row_exponent(top, e):
    x = np.array([[0.0, -top, top / 2, np.nan, np.inf]])
    assert OQ.row_exponents(x)[0] == e


def test_stored_values_are_near_and_are_bf16():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 32)) * 2.0 ** rng.integers(-6, 6, (64, 1))
    bits = OQ.bf16_bits(torch.from_numpy(x).to(torch.bfloat16).double().numpy())
    codes, exps = OQ.quantise(bits)
    v, x = OQ.values(codes, exps), OQ.bf16_values(bits)
    step = 2.0 ** (exps.astype(np.int64)[:, None] - 127.0 - 10)  # half of the smallest step
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step)).all()
    OQ.bf16_bits(v)  # asserts that bf16 holds them


# ----------------------------------------------------------------- refusals
F = 1 << 20  # an address that no call dereferences: every case fails a check first


def write_args(**kw):
    a = dict(k=F, v=F, ks=256, vs=256, slots=F, T=4, kc=F, vc=F, ke=F, ve=F, NB=8, bs=16, Hkv=2, d=128, st=None,
             stream=None)
    a.update(kw)
    return list(a.values())


def read_args(**kw):
    a = dict(kc=F, vc=F, ke=F, ve=F, slots=F, T=4, k=F, v=F, NB=8, bs=16, Hkv=2, d=128, st=None, stream=None)
    a.update(kw)
    return list(a.values())


def decode_args(**kw):
    a = dict(q=F, kc=F, vc=F, ke=F, ve=F, tbl=F, maxb=4, lens=F, B=2, maxlen=64, Hq=8, Hkv=2, d=128, bs=16, NB=8,
             scale=0.1, out=F, ws=None, wsb=0, st=None, stream=None)
    a.update(kw)
    return list(a.values())


ARG, UNSUPPORTED, WORKSPACE = -1, -4, -8
ROWS_BAD = [(dict(T=-1), ARG), (dict(NB=-1), ARG), (dict(bs=0), ARG), (dict(Hkv=0), ARG), (dict(d=0), ARG),
            (dict(d=24), UNSUPPORTED), (dict(d=528), UNSUPPORTED), (dict(k=None), ARG), (dict(v=None), ARG),
            (dict(slots=None), ARG), (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(ke=None), ARG),
            (dict(ve=None), ARG), (dict(k=F + 8), ARG), (dict(v=F + 2), ARG), (dict(kc=F + 4), ARG),
            (dict(vc=F + 1), ARG), (dict(slots=F + 4), ARG)]


@pytest.mark.parametrize("kw,rc", ROWS_BAD + [(dict(ks=255), ARG), (dict(vs=248), ARG), (dict(ks=260), ARG),
                                              (dict(vs=0), ARG), (dict(ks=-256), ARG)])
def test_write_refuses(native, kw, rc):
    assert native.lib().pkv_write_quant(*write_args(**kw)) == rc


@pytest.mark.parametrize("kw,rc", ROWS_BAD)
def test_read_refuses(native, kw, rc):
    assert native.lib().pkv_read_quant(*read_args(**kw)) == rc


def test_no_tokens_is_a_no_op(native):
    assert native.lib().pkv_write_quant(*write_args(T=0, k=None, slots=None)) == 0
    assert native.lib().pkv_read_quant(*read_args(T=0, k=None, slots=None)) == 0
    assert native.lib().paged_attention_decode_quant(*decode_args(B=0, q=None)) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), ARG), (dict(maxb=-1), ARG), (dict(maxlen=-1), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG),
    (dict(NB=-1), ARG), (dict(NB=0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(Hq=7), ARG), (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(bs=48), UNSUPPORTED),
    (dict(Hq=34), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(q=None), ARG), (dict(kc=None), ARG),
    (dict(vc=None), ARG), (dict(ke=None), ARG), (dict(ve=None), ARG), (dict(tbl=None), ARG), (dict(lens=None), ARG),
    (dict(out=None), ARG), (dict(q=F + 8), ARG), (dict(kc=F + 8), ARG), (dict(ke=F + 8), ARG), (dict(out=F + 2), ARG),
    (dict(tbl=F + 2), ARG), (dict(lens=F + 1), ARG), (dict(NB=1 << 27), UNSUPPORTED),
])
def test_decode_refuses(native, kw, rc):
    assert native.lib().paged_attention_decode_quant(*decode_args(**kw)) == rc


def test_decode_refuses_a_missing_or_small_workspace(native):
    n = native.paged_attention_decode_quant_workspace_size(2, 8, 2, 128, 100000)
    if n == 0:
        pytest.skip("these sizes need no workspace")
    kw = dict(maxlen=100000, maxb=10000)
    f = native.lib().paged_attention_decode_quant
    assert f(*decode_args(**kw)) == WORKSPACE
    assert f(*decode_args(ws=F, wsb=n - 1, **kw)) == WORKSPACE
    assert f(*decode_args(ws=F + 8, wsb=n, **kw)) == WORKSPACE


def test_workspace_size_of_invalid_sizes_is_zero(native):
    f = native.paged_attention_decode_quant_workspace_size
    for bad in ((-1, 8, 2, 128, 64), (2, 0, 2, 128, 64), (2, 8, 0, 128, 64), (2, 8, 3, 128, 64), (2, 8, 2, 96, 64),
                (2, 8, 2, 128, -1), (2, 64, 2, 128, 64), (0, 8, 2, 128, 64)):
        assert f(*bad) == 0, bad


def test_workspace_size_never_shrinks_and_may_jump(native):
    """A buffer sized for the largest batch and bound serves every smaller one; one sequence or token
    more may take the need from none to the full size."""
    f = native.paged_attention_decode_quant_workspace_size
    batches = [1, 2, 7, 18, 19, 20, 21, 76, 77, 152, 153, 154, 400, 1672, 1673, 13000, 13377, 65535]
    bounds = [0, 1, 32, 33, 64, 65, 128, 129, 350, 352, 353, 384, 385, 704, 705, 768, 769, 1536, 1537, 5000, 100000]
    for d, Hkv, G in [(128, 8, 4), (128, 1, 8), (128, 2, 16), (64, 3, 1), (64, 4, 12), (64, 16, 8)]:
        size = np.array([[f(b, Hkv * G, Hkv, d, n) for n in bounds] for b in batches], dtype=np.int64)
        assert (np.diff(size, axis=0) >= 0).all() and (np.diff(size, axis=1) >= 0).all()
        assert size[0, 0] == 0
    assert f(400, 32, 8, 128, 352) == 0 and f(400, 32, 8, 128, 353) > 1 << 20
    assert f(152, 8, 1, 128, 704) == 0 and f(153, 8, 1, 128, 704) > 0
    assert f(400, 32, 8, 128, 9000) < 1.3e6 < 2.5e6 < f(400, 128, 8, 128, 9000) < 2.6e6


def cpu_cache(NB=4, Hkv=2, bs=16, d=64):
    c = lambda: torch.zeros((NB, Hkv, bs, d), dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    e = lambda: torch.zeros((NB, Hkv, bs), dtype=torch.uint8)  # noqa: E731
    return [c(), c(), e(), e()]


def test_python_checks_shapes_types_and_devices(native):
    slots, kv = torch.zeros(3, dtype=torch.int64), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    cache = cpu_cache()
    with pytest.raises(ValueError, match="CUDA"):
        native.pkv_write_quant(kv, kv, slots, *cache)
    with pytest.raises(ValueError, match="CUDA"):
        native.pkv_read_quant(*cache, slots, kv, kv.clone())
    with pytest.raises(TypeError):
        native.pkv_write_quant(kv.float(), kv, slots, *cache)
    with pytest.raises(TypeError):
        native.pkv_write_quant(kv, kv, slots.int(), *cache)
    with pytest.raises(TypeError):
        native.pkv_write_quant(kv, kv, slots, cache[0].view(torch.uint8), *cache[1:])
    with pytest.raises(TypeError):
        native.pkv_write_quant(kv, kv, slots, cache[0], cache[1], cache[2].int(), cache[3])
    with pytest.raises(ValueError):
        native.pkv_write_quant(kv[:2], kv, slots, *cache)
    with pytest.raises(ValueError):
        native.pkv_write_quant(kv, kv, slots, cache[0], cache[1], cache[2][:3], cache[3])
    with pytest.raises(ValueError, match="rows must be dense"):
        native.pkv_write_quant(kv[:1].expand(3, 2, 64), kv, slots, *cache)
    with pytest.raises(ValueError, match="rows must be dense"):
        native.pkv_write_quant(kv, torch.zeros((3, 64, 2), dtype=torch.bfloat16).transpose(1, 2), slots, *cache)
    with pytest.raises(ValueError, match="rows must be dense"):  # tokens 132 elements apart
        native.pkv_write_quant(kv, torch.zeros((3, 132), dtype=torch.bfloat16)[:, :128].view(3, 2, 64), slots, *cache)
    with pytest.raises(ValueError):
        native.pkv_read_quant(*cache, slots, kv.transpose(0, 1).contiguous().transpose(0, 1), kv)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    tbl, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        native.paged_attention_decode_quant(q, *cache, tbl, lens, 8, 0.1, q.clone())
    for bad in (q[:, 0], q[:1], q.expand(2, 2, 4, 64).contiguous(), q[..., :32].contiguous()):
        with pytest.raises(ValueError):
            native.paged_attention_decode_quant(bad, *cache, tbl, lens, 8, 0.1, bad.clone())
    with pytest.raises(ValueError):
        native.paged_attention_decode_quant(q, *cache, tbl[:1], lens, 8, 0.1, q.clone())
    with pytest.raises(TypeError):
        native.paged_attention_decode_quant(q, *cache, tbl.long(), lens, 8, 0.1, q.clone())




def test_python_says_what_is_not_a_tensor(native):
    slots, kv = torch.zeros(3, dtype=torch.int64), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    cache = cpu_cache()
    with pytest.raises(TypeError, match="v_codes must be a torch.Tensor"):
        native.pkv_write_quant(kv, kv, slots, cache[0], None, *cache[2:])
    with pytest.raises(TypeError, match="slot_mapping must be a torch.Tensor"):
        native.pkv_write_quant(kv, kv, [0, 1, 2], *cache)
    with pytest.raises(TypeError, match="k must be"):
        native.pkv_write_quant(None, kv, slots, *cache)
    with pytest.raises(TypeError, match="v must be a torch.Tensor"):
        native.pkv_read_quant(*cache, slots, kv, 3)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    tbl, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="seq_lens must be a torch.Tensor"):
        native.paged_attention_decode_quant(q, *cache, tbl, None, 8, 0.1, q.clone())
    with pytest.raises(TypeError, match="d_status"):
        native.paged_attention_decode_quant(q, *cache, tbl, lens, 8, 0.1, q.clone(), None, torch.zeros(1))


def test_decode_oracle_against_a_plain_loop():
    rng = np.random.default_rng(0)
    B, Hkv, G, d, bs, NB, scale = 3, 2, 3, 16, 4, 9, 0.1
    kc, vc = (rng.integers(0, 127, (NB, Hkv, bs, d)).astype(np.uint8) for _ in range(2))
    ke, ve = (rng.integers(110, 120, (NB, Hkv, bs)).astype(np.uint8) for _ in range(2))
    q = np.round(rng.standard_normal((B, Hkv * G, d)) * 8) / 8
    lens, tables = [5, 0, 11], np.array([rng.permutation(NB)[:3] for _ in range(B)])
    out = OQ.decode(OQ.bf16_bits(q), kc, vc, ke, ve, tables, lens, scale)[0]
    for i in range(B):
        for g in range(Hkv * G):
            h, num, den = g // G, np.zeros(d), 0.0
            for t in range(lens[i]):
                b, o = tables[i][t // bs], t % bs
                w = np.exp(scale * 2.0 ** (int(ke[b, h, o]) - 127) * (q[i, g] @ OQ.TABLE[kc[b, h, o]]))
                num, den = num + w * OQ.TABLE[vc[b, h, o]] * 2.0 ** (int(ve[b, h, o]) - 127), den + w
            assert np.allclose(out[i, g], num / den if den else 0.0, rtol=1e-12)
