"""The rotary append on the GPU against the oracle, bit for bit: every product and
sum of the rotation is rounded to fp32, the result once to bf16 (or quantised), so
there is one right answer.  Against float64 the rotation's own error is at most
2^-24 (|a c| + |b s|) for each product and as much for the sum (2^-24 |result|),
then half a bf16 step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from oracle import quant as OQ
from oracle import rope as OR
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


def u8(t):
    return t.detach().contiguous().cpu().view(torch.uint8).numpy().copy()


def gpu_bf16(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).cuda().view(torch.bfloat16)


def status_tensor():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def same_bf16(got, want, exact_from=None):
    """Equal bit patterns; NaN is NaN where the rotation made it."""
    nan = np.isnan(OQ.bf16_values(want))
    ok = (got == want) | (nan & np.isnan(OQ.bf16_values(got)))
    return ok.all()


def rows(T, H, d, rng, awkward):
    """bf16 rows: ordinary ones, or (every third token) any bit pattern, zeros, infinities and NaN."""
    b = bits(torch.from_numpy(rng.standard_normal((T, H, d))).to(torch.bfloat16)).copy()
    if awkward:
        for t in range(0, T, 3):
            kind = (t // 3) % 4
            b[t] = {0: rng.integers(0, 1 << 16, (H, d)), 1: rng.choice([0x0000, 0x8000], (H, d)),
                    2: rng.choice([0x7F80, 0xFF80, 0x7FC0, 0x3F80], (H, d)),
                    3: rng.integers(0, 0x7F80, (H, d))}[kind]
    return b.astype(np.uint16)


def cache(quant, NB, Hkv, bs, d):
    """Untouched slots keep this byte."""
    if not quant:
        return [torch.full((NB, Hkv, bs, d, 2), 0xAB, dtype=torch.uint8, device="cuda").view(torch.bfloat16)[..., 0]
                for _ in "kv"]
    c = [torch.full((NB, Hkv, bs, d), 0xAB, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"]
    return c + [torch.full((NB, Hkv, bs), 0xAB, dtype=torch.uint8, device="cuda") for _ in "kv"]


def expect(qb, kb, vb, pos, cs, slots, inter, host, quant):
    """Oracle: (rotated query bits or None, cache arrays after the call).  Tokens at bad positions write nothing,
    tokens at bad or negative slots only their queries."""
    good = (pos >= 0) & (pos < len(cs))
    p = np.where(good, pos, 0)
    rot = cs.shape[1]

    def turn(b):  # bf16 bits of the rotated rows; the rest keeps its bits
        y = OR.to_bf16(OR.rotate(OQ.bf16_values(b).astype(np.float32), cs, p, inter))
        return np.concatenate([y[..., :rot], b[..., rot:]], -1)

    bs, n = host[0].shape[2], host[0].shape[0] * host[0].shape[2]
    keep = [t for t in range(len(pos)) if good[t] and 0 <= slots[t] < n]
    b, o = slots[keep] // bs, slots[keep] % bs
    if quant:
        kr = OR.rotate(OQ.bf16_values(kb).astype(np.float32), cs, p, inter)
        kc, ke = OR.quantise(kr[keep])
        vc, ve = OQ.quantise(vb[keep])
        for arr, x in zip(host, (kc, vc, ke, ve)):
            arr[b, :, o] = x
    else:
        for arr, x in zip(host, (turn(kb), vb)):
            arr[b, :, o] = x[keep]
    return (None if qb is None else turn(qb)), good, host


CASES = [  # T, Hq, Hkv, d, rot, bs
    (1, 4, 2, 64, 64, 16), (3, 1, 1, 16, 16, 1), (257, 8, 2, 128, 128, 16), (100, 5, 5, 48, 32, 7), (33, 7, 1, 80, 16, 24),
    (65, 6, 3, 96, 96, 32), (41, 3, 1, 112, 48, 128), (20, 4, 4, 192, 160, 64), (19, 2, 1, 256, 256, 8), (9, 3, 2, 512, 496, 16),
    (1031, 32, 8, 128, 64, 16), (50, 0, 3, 64, 32, 16), (5, 16, 1, 32, 32, 16), (7, 2, 1, 528 - 16, 512, 4),
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,bs", CASES)
def test_bit_exact(T, Hq, Hkv, d, rot, bs, interleaved, quant):
    rng = np.random.default_rng(T + 5 * d + rot)
    NB = -(-2 * T // bs) + 3
    top = 200
    cs = OR.table(top, rot)
    pos = rng.integers(0, top, T)
    slots = inputs.distinct_slots(T, NB * bs, rng, skip_fraction=0.2 if T > 1 else 0.0)
    qb = rows(T, Hq, d, rng, T > 4) if Hq else None
    kb, vb = rows(T, Hkv, d, rng, T > 4), rows(T, Hkv, d, rng, T > 4)
    c = cache(quant, NB, Hkv, bs, d)
    host = [u8(t) if quant else bits(t).copy() for t in c]
    want_q, _, want = expect(qb, kb, vb, pos, cs, slots, interleaved, host, quant)
    q = gpu_bf16(qb) if Hq else None
    out = torch.zeros_like(q) if Hq else None
    st = status_tensor()
    f = native.pkv_write_rope_quant if quant else native.pkv_write_rope
    f(q, gpu_bf16(kb), gpu_bf16(vb), torch.from_numpy(pos).cuda(), torch.from_numpy(cs).cuda(),
      torch.from_numpy(slots).cuda(), out, *c, interleaved=interleaved, d_status=st)
    assert st.item() == 0
    if Hq:
        assert same_bf16(bits(out), want_q)
    for t, w in zip(c, want):
        assert np.array_equal(u8(t), w) if quant else same_bf16(bits(t), w)


def test_near_the_float64_rotation():
    rng = np.random.default_rng(5)
    T, H, d, rot = 64, 4, 128, 128
    cs = OR.table(131072, rot)
    pos = rng.integers(100000, 131072, T)
    xb = rows(T, H, d, rng, False)
    q, c = gpu_bf16(xb), cache(False, T, H, 1, d)
    out = torch.zeros_like(q)
    native.pkv_write_rope(q, q, q, torch.from_numpy(pos).cuda(), torch.from_numpy(cs).cuda(),
                          torch.arange(T, device="cuda"), out, *c)
    x = OQ.bf16_values(xb)
    want = OR.rotate(x, cs, pos, False, np.float64)
    i, j = OR.pairs(rot, False)
    size = np.hypot(x[..., i], x[..., j])  # >= |a c| + |b s| over sqrt(2)
    bound = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8)
    bound[..., i] += 2.0 ** -23 * 2 ** 0.5 * size
    bound[..., j] += 2.0 ** -23 * 2 ** 0.5 * size
    for got in (OQ.bf16_values(bits(out)), OQ.bf16_values(bits(c[0])[:, :, 0])):
        assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("lie", ["fused", "fused_in_place", "in_place", "odd_rows"])
def test_rows_that_lie_differently(lie, quant):
    rng = np.random.default_rng(11)
    T, Hq, Hkv, d, rot, bs, NB = 77, 6, 2, 64, 48, 16, 12
    cs, pos = OR.table(90, rot), rng.integers(0, 90, T)
    slots = inputs.distinct_slots(T, NB * bs, rng, skip_fraction=0.1)
    qb, kb, vb = (rows(T, h, d, rng, True) for h in (Hq, Hkv, Hkv))
    c = cache(quant, NB, Hkv, bs, d)
    host = [u8(t) if quant else bits(t).copy() for t in c]
    want_q, _, want = expect(qb, kb, vb, pos, cs, slots, True, host, quant)
    pad = 8 if lie == "odd_rows" else 0  # token strides that are odd multiples of 16 bytes
    fused = torch.zeros((T, (Hq + 2 * Hkv) * d + pad), dtype=torch.bfloat16, device="cuda")
    views = [fused[:, a * d:(a + h) * d].unflatten(1, (h, d)) for a, h in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv))]
    for v, b in zip(views, (qb, kb, vb)):
        v.copy_(gpu_bf16(b))
    q, k, v = views if lie != "in_place" else [x.contiguous() for x in views]
    out = q if lie in ("in_place", "fused_in_place") else torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    f = native.pkv_write_rope_quant if quant else native.pkv_write_rope
    f(q, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(cs).cuda(), torch.from_numpy(slots).cuda(), out, *c,
      interleaved=True)
    assert same_bf16(bits(out), want_q)
    assert same_bf16(bits(k), kb) and same_bf16(bits(v), vb)
    for t, w in zip(c, want):
        assert np.array_equal(u8(t), w) if quant else same_bf16(bits(t), w)


@pytest.mark.parametrize("quant", [False, True])
def test_bad_positions_and_slots_are_reported(quant):
    rng = np.random.default_rng(12)
    T, Hq, Hkv, d, rot, bs, NB = 9, 3, 2, 32, 16, 4, 5
    cs = OR.table(30, rot)
    qb, kb, vb = (rows(T, h, d, rng, False) for h in (Hq, Hkv, Hkv))
    slots = np.array([0, 5, NB * bs, 7, -1, 1 << 40, 9, 2, 3])
    for pos, bit in ((np.array([0, 30, 1, 2, -1, 3, 1 << 40, 4, 29]), 64 | 1),
                     (np.array([0, 29, 1, 2, 5, 3, 9, 4, 29]), 1)):
        c = cache(quant, NB, Hkv, bs, d)
        host = [u8(t) if quant else bits(t).copy() for t in c]
        want_q, good, want = expect(qb, kb, vb, pos, cs, slots, False, host, quant)
        out, st = gpu_bf16(np.full((T, Hq, d), 0xABAB, np.uint16)), status_tensor()
        f = native.pkv_write_rope_quant if quant else native.pkv_write_rope
        f(gpu_bf16(qb), gpu_bf16(kb), gpu_bf16(vb), torch.from_numpy(pos).cuda(), torch.from_numpy(cs).cuda(),
          torch.from_numpy(slots).cuda(), out, *c, d_status=st)
        assert st.item() == bit
        got = bits(out)
        assert same_bf16(got[good], want_q[good]) and (got[~good] == 0xABAB).all()
        for t, w in zip(c, want):
            assert np.array_equal(u8(t), w) if quant else same_bf16(bits(t), w)


def test_the_8_bit_append_of_a_zero_rotation_is_the_quantising_write():
    """At position 0 nothing turns: the same codes and exponents as pkv_write_quant's."""
    rng = np.random.default_rng(13)
    T, Hkv, d, bs, NB = 60, 3, 128, 16, 6
    kb, vb = rows(T, Hkv, d, rng, False), rows(T, Hkv, d, rng, False)
    a, b = cache(True, NB, Hkv, bs, d), cache(True, NB, Hkv, bs, d)
    slots = torch.from_numpy(inputs.distinct_slots(T, NB * bs, rng)).cuda()
    native.pkv_write_quant(gpu_bf16(kb), gpu_bf16(vb), slots, *a)
    native.pkv_write_rope_quant(None, gpu_bf16(kb), gpu_bf16(vb), torch.zeros_like(slots),
                                torch.from_numpy(OR.table(4, d)).cuda(), slots, None, *b)
    for x, y in zip(a, b):
        assert np.array_equal(u8(x), u8(y))


def test_captured_and_replayed_on_another_stream():
    rng = np.random.default_rng(14)
    T, Hq, Hkv, d, bs, NB = 40, 4, 2, 64, 16, 8
    cs = OR.table(64, d)
    q, k, v = (torch.zeros((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    pos, slots = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.arange(T, device="cuda")
    table, out = torch.from_numpy(cs).cuda(), torch.zeros_like(q)
    c = cache(False, NB, Hkv, bs, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        native.pkv_write_rope(q, k, v, pos, table, slots, out, *c)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        native.pkv_write_rope(q, k, v, pos, table, slots, out, *c)
    for _ in range(2):
        qb, kb, vb = (rows(T, h, d, rng, False) for h in (Hq, Hkv, Hkv))
        p, s = rng.integers(0, 64, T), rng.permutation(NB * bs)[:T]
        for t, x in ((q, gpu_bf16(qb)), (k, gpu_bf16(kb)), (v, gpu_bf16(vb)), (pos, torch.from_numpy(p).cuda()),
                     (slots, torch.from_numpy(s).cuda())):
            t.copy_(x)
        host = [bits(t).copy() for t in c]
        want_q, _, want = expect(qb, kb, vb, p, cs, s, False, host, False)
        g.replay()
        torch.cuda.synchronize()
        assert same_bf16(bits(out), want_q)
        assert all(same_bf16(bits(t), w) for t, w in zip(c, want))


def test_offsets_past_32_bits():
    """Rows and slots beyond 4 GiB of the cache and of a strided projection's output."""
    Hkv, d, bs = 8, 128, 16
    NB = (1 << 33) // (Hkv * d * bs * 2) + 3  # 8 GiB per array
    kc = torch.zeros((NB, Hkv, bs, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    stride = (1 << 32) // 3 // 16 * 16 + 16  # elements: the last token lies beyond 2^32 elements
    buf = torch.zeros(3 * stride + 2 * Hkv * d, dtype=torch.bfloat16, device="cuda")
    view = buf.as_strided((4, Hkv, d), (stride, d, 1))
    rng = np.random.default_rng(15)
    b = rows(4, Hkv, d, rng, False)
    view.copy_(gpu_bf16(b))
    slots = np.array([NB * bs - 1, 3, NB * bs - 40, NB * bs // 2])
    pos = np.array([1, 9, 30, 0])
    cs = OR.table(31, 64)
    out = torch.zeros((4, Hkv, d), dtype=torch.bfloat16, device="cuda")
    st = status_tensor()
    native.pkv_write_rope(view, view, view, torch.from_numpy(pos).cuda(), torch.from_numpy(cs).cuda(),
                          torch.from_numpy(slots).cuda(), out, kc, vc, d_status=st)
    assert st.item() == 0
    turned = OR.to_bf16(OR.rotate(OQ.bf16_values(b).astype(np.float32), cs, pos, False))
    assert same_bf16(bits(out), turned)
    for t, s in enumerate(slots.tolist()):
        assert same_bf16(bits(kc[s // bs, :, s % bs]), turned[t])
        assert same_bf16(bits(vc[s // bs, :, s % bs]), b[t])
    assert int((vc != 0).any(-1).sum()) == 4 * Hkv
