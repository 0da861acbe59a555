"""The 8-bit cache on the GPU against the float64 oracle: the quantising write and
the read-back bit for bit, the decode within a bound derived below.

Decode bound.  With s the logits, p the weights, A = max_t scale sum_i |q_i k_ti|,
mag = sum_t p_t |v_t| (per output value), n keys:
  * logits: q and the codes enter their products exactly; n_d = d products summed
    in fp32, each addition off by at most 2^-23 of a partial sum <= A, and a few
    roundings of the scaling and of the exponent's argument: (d + 16) 2^-23 A;
    each weight is then off by that relatively, and so is the sum of the weights;
  * 2^x of the hardware and the final division: 2^-20;
  * weights are rounded to 11 significant bits for the product with the values:
    2^-11; weights far below the largest lose bits absolutely, at most 2^-32 of
    the largest weight times value scale, per key, times a code of at most 448;
  * fp32 sums over n keys, of weights and of products: 2 n 2^-24;
  * the output's rounding to bf16: 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import quant as OQ
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


def status_tensor():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def dev(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda").to(dtype)


def cache_on_gpu(kc, vc, ke, ve):
    f8 = torch.float8_e4m3fn
    return [torch.from_numpy(kc).cuda().view(f8), torch.from_numpy(vc).cuda().view(f8), torch.from_numpy(ke).cuda(),
            torch.from_numpy(ve).cuda()]


def random_cache(NB, Hkv, bs, d, rng, fill=None):
    """Host cache arrays: quantised N(0, 1) rows of several sizes, or one byte throughout."""
    if fill is not None:
        return [np.full((NB, Hkv, bs, d), fill, np.uint8), np.full((NB, Hkv, bs, d), fill, np.uint8),
                np.full((NB, Hkv, bs), fill, np.uint8), np.full((NB, Hkv, bs), fill, np.uint8)]
    out = []
    for _ in range(2):
        x = rng.standard_normal((NB, Hkv, bs, d)) * 2.0 ** rng.integers(-2, 3, (NB, Hkv, bs, 1))
        x = torch.from_numpy(x).to(torch.bfloat16)
        out.append(OQ.quantise(bits(x)))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


# ---------------------------------------------------------------------- write
def awkward_rows(T, Hkv, d, rng):
    """bf16 bit patterns: ordinary rows, all sizes of the type, ties, zeros, NaN and infinities."""
    x = torch.from_numpy(rng.standard_normal((T, Hkv, d))).to(torch.bfloat16)
    b = bits(x).copy()
    kinds = rng.integers(0, 9, (T, Hkv))
    for t in range(T):
        for h in range(Hkv):
            r, kind = b[t, h], kinds[t, h]
            if kind == 1:    # any bit pattern at all
                r[:] = rng.integers(0, 1 << 16, d)
            elif kind == 2:  # zeros of both signs
                r[:] = rng.choice([0x0000, 0x8000], d)
            elif kind == 3:  # subnormal and tiny values
                r[:] = rng.integers(0, 0x0200, d)
            elif kind == 4:  # finite values of every size
                r[:] = rng.integers(0, 0x7F80, d) | rng.choice([0, 0x8000], d)
            elif kind == 5:  # a row's largest at, just above and just below 448 * 2^e, and halves of code steps
                e = int(rng.integers(-20, 20))
                vals = np.array([448.0, 450.0, 446.0, 1.0625, 1.1875, 1.3125, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9])
                r[:] = OQ.bf16_bits(rng.choice(vals[int(rng.integers(0, 3)):], d) * 2.0 ** e)
            elif kind == 6:  # one NaN or infinity among ordinary values
                r[int(rng.integers(0, d))] = rng.choice([0x7FC0, 0xFFC1, 0x7F80, 0xFF80, 0x7F81])
            elif kind == 7:  # one value far above the others
                r[int(rng.integers(0, d))] = 0x4800
            elif kind == 8 and rng.random() < 0.3:
                r[:] = 0x7F80
    return b


def gpu_bf16(b):
    return torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16)


@pytest.mark.parametrize("T,Hkv,d,bs,strided", [
    (1, 1, 16, 1, False), (300, 8, 128, 16, False), (257, 2, 64, 32, True), (33, 3, 48, 7, True), (40, 5, 80, 24, False),
    (64, 1, 96, 128, True), (21, 2, 112, 16, False), (19, 4, 192, 8, True), (17, 3, 256, 64, False), (9, 2, 512, 16, True),
    (1, 8, 128, 16, True), (5000, 1, 32, 16, False), (5003, 8, 128, 16, True), (4999, 9, 64, 64, False),
])
def test_write_bit_exact(T, Hkv, d, bs, strided):
    rng = np.random.default_rng(T + 7 * d + bs)
    NB = -(-2 * T // bs) + 3
    slots = inputs.distinct_slots(T, NB * bs, rng, skip_fraction=0.1 if T > 1 else 0.0)
    kb, vb = awkward_rows(T, Hkv, d, rng), awkward_rows(T, Hkv, d, rng)
    host = random_cache(NB, Hkv, bs, d, rng, fill=0xAB)  # untouched slots keep this byte
    cache = cache_on_gpu(*[a.copy() for a in host])
    if strided:  # the key and value columns of one projection's output
        fused = torch.zeros((T, Hkv * d * 3 + 16), dtype=torch.bfloat16, device="cuda")
        k = fused[:, 8:8 + Hkv * d].view(T, Hkv, d) if T > 1 else fused[:, 8:8 + Hkv * d].reshape(T, Hkv, d)
        v = fused[:, 16 + Hkv * d:16 + 2 * Hkv * d].view(T, Hkv, d)
        k.copy_(gpu_bf16(kb))
        v.copy_(gpu_bf16(vb))
    else:
        k, v = gpu_bf16(kb), gpu_bf16(vb)
    OQ.write(kb, vb, slots, *host)
    st = status_tensor()
    native.pkv_write_quant(k, v, dev(slots, torch.int64), *cache, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for got, want, what in zip(cache, host, ("key codes", "value codes", "key exponents", "value exponents")):
        g = u8(got)
        assert np.array_equal(g, want), f"{what}: {int((g != want).sum())} of {want.size} differ"


def test_rows_aligned_to_16_bytes_only():
    """Buffers 16 bytes off a 32-byte boundary, for the write's input and the read-back's output."""
    T, Hkv, d, bs = 300, 3, 64, 16
    rng = np.random.default_rng(12)
    host = random_cache(40, Hkv, bs, d, rng, fill=0)
    cache = cache_on_gpu(*[a.copy() for a in host])
    slots = inputs.distinct_slots(T, 40 * bs, rng)
    kb, vb = awkward_rows(T, Hkv, d, rng), awkward_rows(T, Hkv, d, rng)

    def off16(b=None):
        t = torch.zeros(T * Hkv * d + 16, dtype=torch.bfloat16, device="cuda")
        t = t[8:8 + T * Hkv * d] if t.data_ptr() % 32 == 0 else t[:T * Hkv * d]
        t = t.view(T, Hkv, d)
        assert t.data_ptr() % 32 == 16
        return t if b is None else t.copy_(gpu_bf16(b))

    native.pkv_write_quant(off16(kb), off16(vb), dev(slots, torch.int64), *cache)
    OQ.write(kb, vb, slots, *host)
    k, v = off16(), off16()
    native.pkv_read_quant(*cache, dev(slots, torch.int64), k, v)
    torch.cuda.synchronize()
    assert all(np.array_equal(u8(g), w) for g, w in zip(cache, host))
    for got, codes, exps in ((k, host[0], host[2]), (v, host[1], host[3])):
        want = OQ.values(codes[slots // bs, :, slots % bs], exps[slots // bs, :, slots % bs])
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


def test_write_out_of_range_slots_are_reported_and_skipped():
    rng = np.random.default_rng(0)
    NB, Hkv, bs, d = 4, 2, 16, 64
    host = random_cache(NB, Hkv, bs, d, rng, fill=0x11)
    cache = cache_on_gpu(*[a.copy() for a in host])
    kb = awkward_rows(4, Hkv, d, rng)
    st = status_tensor()
    native.pkv_write_quant(gpu_bf16(kb), gpu_bf16(kb), dev([5, NB * bs, -3, 1 << 62], torch.int64), *cache, st)
    torch.cuda.synchronize()
    assert st.item() == native.PKV_STATUS_BAD_SLOT
    OQ.write(kb[:1], kb[:1], [5], *host)
    assert all(np.array_equal(u8(g), w) for g, w in zip(cache, host))


# ------------------------------------------------------------------- read back
@pytest.mark.parametrize("T,Hkv,d,bs", [(1, 1, 16, 1), (700, 8, 128, 16), (65, 3, 48, 7), (31, 2, 512, 32), (90, 5, 80, 24)])
def test_read_back_is_exact(T, Hkv, d, bs):
    rng = np.random.default_rng(T + d)
    NB = max(3, T // (2 * bs))
    host = [rng.integers(0, 256, (NB, Hkv, bs, d)).astype(np.uint8) for _ in range(2)] + \
           [rng.integers(0, 256, (NB, Hkv, bs)).astype(np.uint8) for _ in range(2)]  # every byte there is
    slots = rng.integers(0, NB * bs, T).astype(np.int64)  # repeated slots
    slots[rng.random(T) < 0.1] = -1
    k = torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((T, Hkv, d), -7.0, dtype=torch.bfloat16, device="cuda")
    st = status_tensor()
    native.pkv_read_quant(*cache_on_gpu(*host), dev(slots, torch.int64), k, v, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for got, codes, exps, keep in ((k, host[0], host[2], 7.0), (v, host[1], host[3], -7.0)):
        want = np.full((T, Hkv, d), keep)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                want[t] = OQ.values(codes[s // bs, :, s % bs], exps[s // bs, :, s % bs])
        g = got.double().cpu().numpy()
        assert np.array_equal(g, want, equal_nan=True)


def test_read_back_reports_slots_past_the_pool_and_leaves_their_rows():
    rng = np.random.default_rng(1)
    host = random_cache(3, 2, 16, 64, rng)
    k = torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    v, st = k.clone(), status_tensor()
    native.pkv_read_quant(*cache_on_gpu(*host), dev([48, 3, 1 << 40], torch.int64), k, v, st)
    torch.cuda.synchronize()
    assert st.item() == native.PKV_STATUS_BAD_SLOT
    assert (k[[0, 2]] == 5.0).all() and (v[[0, 2]] == 5.0).all()
    assert np.array_equal(k[1].double().cpu().numpy(), OQ.values(host[0][0, :, 3], host[2][0, :, 3]))


# --------------------------------------------------------------------- decode
def workspace_for(B, Hq, Hkv, d, max_len):
    n = native.paged_attention_decode_quant_workspace_size(B, Hq, Hkv, d, max_len)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # NaN patterns: nothing may be read before it is written
    return ws


def run_decode(q, cache, tables, lens, scale, max_len=None, status=None, ws=None, stream=None):
    B, _, Hq, d = q.shape
    max_len = int(np.max(lens, initial=0)) if max_len is None else max_len
    ws = workspace_for(B, Hq, cache[0].shape[1], d, max_len) if ws is None else ws
    out = torch.full_like(q, float("nan"))
    native.paged_attention_decode_quant(q, *cache, dev(tables, torch.int32), dev(lens, torch.int32), max_len, scale, out,
                                        ws, status, stream)
    torch.cuda.synchronize()
    return out


def decode_case(lens, d, bs, Hq, Hkv, seed, spare=3):
    rng = np.random.default_rng(seed)
    NB = sum(inputs.entries_to_fill(n, bs) for n in lens) + spare
    tables, _ = inputs.permuted_tables(lens, bs, NB, rng,
                                       max_blocks=max(1, max(inputs.entries_to_fill(n, bs) for n in lens)) + 2)
    host = random_cache(NB, Hkv, bs, d, rng)
    q = torch.from_numpy(rng.standard_normal((len(lens), 1, Hq, d)) * 2.0 ** rng.integers(-3, 3, (len(lens), 1, Hq, 1)))
    return q.to(torch.bfloat16).cuda(), host, tables


def check_decode(out, q, host, tables, lens, scale, what=""):
    d = q.shape[-1]
    ref, mag, dot, top = OQ.decode(bits(q)[:, 0], *host, tables, lens, scale)
    n = np.asarray(lens, dtype=np.float64)[:, None, None]
    weights = 2 * (d + 16) * 2.0 ** -23 * dot[..., None] + 2.0 ** -20 + 2.0 ** -11 + 2 * n * 2.0 ** -24
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (mag * weights + n * 2.0 ** -32 * 448 * top[..., None])
    got = out[:, 0].double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got - ref)
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside the bound; worst {(err / bound)[bad].max():.2f} times it"


ODD = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 0, 255, 700]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_decode_odd_lengths(d, bs):
    q, host, tables = decode_case(ODD, d, bs, 8, 2, seed=d + bs)
    st = status_tensor()
    out = run_decode(q, cache_on_gpu(*host), tables, ODD, d ** -0.5, status=st)
    assert st.item() == 0
    assert not out[15].any()  # no keys: zeros
    check_decode(out, q, host, tables, ODD, d ** -0.5)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (2, 1), (9, 3), (10, 2), (7, 1), (16, 2), (9, 1), (24, 2), (16, 1), (48, 3)])
def test_decode_head_layouts(Hq, Hkv):
    lens = [37, 1, 300, 90]
    for d, bs in ((64, 16), (128, 32)):
        q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=Hq * 17 + d)
        check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, d ** -0.5), q, host, tables, lens, d ** -0.5)


@pytest.mark.parametrize("lens,Hq,Hkv,d,bs", [([20011], 8, 1, 128, 16), ([9000, 5, 12345], 16, 2, 64, 64), ([40000], 4, 4, 64, 128),
                                              ([4097, 4096, 4095, 2049], 32, 4, 128, 16), ([3000] + [40] * 30, 4, 2, 128, 32)])
def test_decode_long_and_mixed_lengths(lens, Hq, Hkv, d, bs):
    q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=sum(lens) % 1000)
    for max_len in (None, max(lens) + 5000):  # the caller's bound may be loose
        check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, d ** -0.5, max_len=max_len), q, host, tables, lens,
                     d ** -0.5)


@pytest.mark.parametrize("lens,Hq,Hkv,d,bs", [([60000], 4, 1, 128, 64), ([70001], 12, 1, 128, 128), ([40000, 0, 33001], 2, 1, 64, 16),
                                              ([50000], 48, 3, 64, 32), ([45000, 1], 21, 3, 128, 16), ([20000], 7, 7, 64, 64)])
def test_decode_few_long_runs(lens, Hq, Hkv, d, bs):
    """A run over up to the whole grid: many pieces to join, with one to seven runs."""
    q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=sum(lens) % 997)
    cache = cache_on_gpu(*host)
    out = run_decode(q, cache, tables, lens, d ** -0.5)
    check_decode(out, q, host, tables, lens, d ** -0.5)
    assert np.array_equal(bits(run_decode(q, cache, tables, lens, d ** -0.5)), bits(out))


def test_decode_many_sequences():
    rng = np.random.default_rng(4)
    lens = np.minimum(rng.geometric(0.03, 3000), 200).astype(np.int64)
    lens[rng.random(3000) < 0.1] = 0
    q, host, tables = decode_case(lens.tolist(), 64, 16, 2, 1, seed=8)
    check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, 0.125), q, host, tables, lens, 0.125)


@pytest.mark.parametrize("d,Hq,Hkv,top", [(128, 6, 3, 384), (128, 6, 3, 385), (64, 4, 2, 768), (64, 4, 2, 769), (128, 24, 2, 256),
                                          (128, 24, 2, 257), (64, 12, 1, 640), (64, 12, 1, 641), (128, 5, 5, 33),
                                          (128, 2, 2, 704), (128, 2, 2, 705), (64, 2, 1, 1536), (64, 2, 1, 1537)])
def test_decode_short_sequences(d, Hq, Hkv, top):
    """Batches around the length up to which no sequence is split between CTAs."""
    rng = np.random.default_rng(top)
    for B in (1, 40, 400 if top < 700 else 160):
        lens = rng.integers(0, top + 1, B)
        lens[rng.integers(0, B, 3)] = top
        q, host, tables = decode_case(lens.tolist(), d, 16, Hq, Hkv, seed=top + B)
        check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, d ** -0.5), q, host, tables, lens, d ** -0.5)


@pytest.mark.parametrize("d,Hq,Hkv,bs,top", [(128, 8, 2, 16, 64), (128, 8, 2, 16, 65), (64, 4, 4, 32, 128), (64, 4, 4, 32, 129),
                                             (128, 16, 1, 128, 64), (64, 12, 1, 64, 128), (128, 3, 3, 64, 1), (64, 1, 1, 16, 33)])
def test_decode_very_short_sequences(d, Hq, Hkv, bs, top):
    """Batches around the length up to which a sequence is one warp's, from one sequence to more runs than warps."""
    rng = np.random.default_rng(top + bs)
    for B in (1, 5, 300, 900 if Hkv > 1 else 2000):
        lens = rng.integers(0, top + 1, B)
        lens[rng.integers(0, B, 3)] = top
        q, host, tables = decode_case(lens.tolist(), d, bs, Hq, Hkv, seed=top + B)
        st = status_tensor()
        out = run_decode(q, cache_on_gpu(*host), tables, lens, d ** -0.5, status=st)
        assert st.item() == 0
        check_decode(out, q, host, tables, lens, d ** -0.5)
        bad = lens.copy()
        bad[0] = -3
        out = run_decode(q, cache_on_gpu(*host), tables, bad, d ** -0.5, max_len=top, status=st)
        assert st.item() == native.PKV_STATUS_BAD_LEN and not out[0].any()


def test_decode_all_empty():
    q, host, tables = decode_case([0, 0, 0], 128, 16, 8, 2, seed=2)
    for max_len in (0, 100, 100000):
        assert not run_decode(q, cache_on_gpu(*host), tables, [0, 0, 0], 0.1, max_len=max_len).any()


@pytest.mark.parametrize("scale", [0.0, -0.3, 8.0])
def test_decode_scales(scale):
    lens = [200, 3, 1000]
    q, host, tables = decode_case(lens, 128, 16, 8, 2, seed=11)
    check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, scale), q, host, tables, lens, scale)


@pytest.mark.parametrize("byte", [0x7F, 0xFF, 0x00])
def test_bytes_behind_a_sequence_never_count(byte):
    """Slots past each end, spare blocks and table entries past a sequence's blocks hold NaN codes,
    exponents of any size and ids of other blocks."""
    lens, bs, d = [1, 15, 33, 90, 200, 0], 64, 128
    q, host, tables = decode_case(lens, d, bs, 8, 2, seed=5)
    used = np.zeros((host[0].shape[0], bs), dtype=bool)
    for i, n in enumerate(lens):
        for t in range(n):
            used[tables[i, t // bs], t % bs] = True
    dirty = [a.copy() for a in host]
    for a in dirty:
        a.swapaxes(0, 1)[:, ~used] = byte
    want = run_decode(q, cache_on_gpu(*host), tables, lens, 0.1)
    wild = tables.copy()
    for i, n in enumerate(lens):
        wild[i, -(-n // bs):] = [7, -5, 1 << 30, 0, 2][i % 5]
    st = status_tensor()
    got = run_decode(q, cache_on_gpu(*dirty), wild, lens, 0.1, status=st)
    assert st.item() == 0
    assert np.array_equal(bits(got), bits(want))
    check_decode(got, q, host, tables, lens, 0.1)


def test_nan_at_a_visible_key_or_value_shows():
    lens, bs, d = [40, 40, 40], 16, 64
    q, host, tables = decode_case(lens, d, bs, 4, 2, seed=6)
    host[0][tables[0, 1], 0, 3, 5] = 0x7F  # a key of sequence 0, head 0
    host[1][tables[1, 2], 1, 7, 9] = 0xFF  # a value of sequence 1, head 1
    out = run_decode(q, cache_on_gpu(*host), tables, lens, 0.125)[:, 0].isnan().cpu().numpy()
    assert out[0, :2].all() and not out[0, 2:].any()
    assert not out[1, :2].any() and out[1, 2:, 9].all() and out[1, 2:].sum() == 2
    assert not out[2].any()


@pytest.mark.parametrize("bound", [40, 5000, 30000])
def test_infinite_queries_show(bound):
    """A query head with an infinity has no finite answer, not even where all its scores are -inf
    (0 / 0); the other heads of its group keep theirs.  The bounds take the three schedules."""
    lens, bs, d = [1, 40, 33], 16, 64
    if bound > 40:
        lens = [1, bound, 700]
    q, host, tables = decode_case(lens, d, bs, 8, 2, seed=16)
    q[:, 0, 1, 0] = float("-inf")
    q[:, 0, 6, 0] = float("inf")
    host[0][..., 0] = 0x38  # every key's first value is positive
    got = run_decode(q, cache_on_gpu(*host), tables, lens, 0.125)[:, 0].double().cpu().numpy()
    assert np.isnan(got[:, [1, 6]]).all()
    rest = [0, 2, 3, 4, 5, 7]
    assert np.isfinite(got[:, rest]).all()
    q[:, 0, [1, 6], 0] = 0.0
    out = run_decode(q, cache_on_gpu(*host), tables, lens, 0.125)
    check_decode(out, q, host, tables, lens, 0.125)
    assert np.array_equal(out[:, 0].double().cpu().numpy()[:, rest], got[:, rest])


def test_values_of_every_size():
    """Rows of values 2^62 apart and zero rows, with the weight on any of them: the weights' sum
    must not lose the keys whose values are small."""
    rng = np.random.default_rng(9)
    lens, bs, d, Hq, Hkv = [64, 200, 37, 1000], 16, 64, 4, 2
    q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=13)
    for a in range(host[3].shape[0]):
        host[3][a] = rng.integers(96, 159, host[3][a].shape)
    zero = rng.random(host[3].shape) < 0.5
    host[1][zero] = 0
    host[3][zero] = 96
    for scale in (0.125, 0.0, 3.0):
        check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, scale), q, host, tables, lens, scale, f"scale {scale}")


def test_keys_of_every_size():
    rng = np.random.default_rng(10)
    lens, bs, d, Hq, Hkv = [64, 200, 37], 16, 64, 4, 2
    q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=14)
    host[2][:] = rng.integers(96, 122, host[2].shape)
    check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, 0.125), q, host, tables, lens, 0.125)


def test_queries_of_every_size():
    """Query heads 2^60 apart in one group, zeros and subnormals among their values."""
    rng = np.random.default_rng(15)
    lens = [64, 130]
    q, host, tables = decode_case(lens, 128, 16, 8, 1, seed=15)
    host[2][:] = 118
    size = 2.0 ** np.array([-100, -30, -8, 0, 1, 2, -126, -3], dtype=np.float64)
    x = rng.standard_normal((2, 1, 8, 128)) * size[None, None, :, None]
    x[:, :, :, ::7] = 0.0
    x[:, :, 3] *= 2.0 ** rng.integers(-40, 1, (2, 1, 128))
    x[1, 0, 5] = 0.0
    q = torch.from_numpy(x).to(torch.bfloat16).cuda()
    check_decode(run_decode(q, cache_on_gpu(*host), tables, lens, 0.3), q, host, tables, lens, 0.3)


def test_bad_lengths_and_blocks_are_reported():
    lens, bs, d = [50, 60, 20], 16, 64
    q, host, tables = decode_case(lens, d, bs, 4, 2, seed=7)
    cache = cache_on_gpu(*host)
    cap = tables.shape[1] * bs
    st = status_tensor()
    out = run_decode(q, cache, tables, [-4, cap + 1, 20], 0.1, max_len=10 * cap, status=st)
    assert st.item() & native.PKV_STATUS_BAD_LEN
    assert not out[0].any()
    st = status_tensor()
    out = run_decode(q, cache, tables, lens, 0.1, max_len=32, status=st)  # lengths above the caller's bound
    assert st.item() == native.PKV_STATUS_BAD_LEN
    check_decode(out, q, host, tables, [32, 32, 20], 0.1)
    for bad in (-1, host[0].shape[0], 1 << 30):  # the block's keys and values read as zeros
        broken = tables.copy()
        broken[1, 1] = bad
        st = status_tensor()
        out = run_decode(q, cache, broken, lens, 0.1, status=st)
        assert st.item() == native.PKV_STATUS_BAD_BLOCK
        zeroed = [np.concatenate([a, np.zeros_like(a[:1])]) for a in host]
        zeroed[2][-1] = zeroed[3][-1] = 127
        broken[1, 1] = host[0].shape[0]
        check_decode(out, q, zeroed, broken, lens, 0.1)


def test_decode_repeats_bit_for_bit():
    lens = [3000, 77, 1500, 1]
    q, host, tables = decode_case(lens, 128, 16, 16, 2, seed=21)
    cache = cache_on_gpu(*host)
    first = bits(run_decode(q, cache, tables, lens, 0.1))
    for _ in range(3):
        assert np.array_equal(bits(run_decode(q, cache, tables, lens, 0.1)), first)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 code bytes; the sequences live at its end, and the write goes there."""
    Hkv, bs, d = 8, 16, 128
    NB = (1 << 32) // (Hkv * bs * d) + 40
    cache = [torch.zeros((NB, Hkv, bs, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)] + \
            [torch.zeros((NB, Hkv, bs), dtype=torch.uint8, device="cuda") for _ in range(2)]
    rng = np.random.default_rng(2)
    lens = [70, 33]
    tables = np.full((2, 5), -1, dtype=np.int32)
    tables[0, :5] = NB - 1 - np.arange(5)
    tables[1, :3] = NB - 20 + np.arange(3)
    slots = np.concatenate([[tables[i, t // bs] * bs + t % bs for t in range(n)] for i, n in enumerate(lens)])
    kb, vb = (bits(torch.from_numpy(rng.standard_normal((103, Hkv, d))).to(torch.bfloat16)) for _ in range(2))
    native.pkv_write_quant(gpu_bf16(kb), gpu_bf16(vb), dev(slots, torch.int64), *cache)
    q = torch.from_numpy(rng.standard_normal((2, 1, 16, d))).to(torch.bfloat16).cuda()
    out = run_decode(q, cache, tables, lens, 0.09)
    k, v = (torch.zeros((103, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    native.pkv_read_quant(*cache, dev(slots, torch.int64), k, v)
    torch.cuda.synchronize()
    low = [np.zeros((60, Hkv, bs, d), np.uint8), np.zeros((60, Hkv, bs, d), np.uint8), np.zeros((60, Hkv, bs), np.uint8),
           np.zeros((60, Hkv, bs), np.uint8)]
    shift = NB - 60
    low_tables = np.where(tables >= 0, tables - shift, -1)
    OQ.write(kb, vb, slots - shift * bs, *low)
    check_decode(out, q, low, low_tables, lens, 0.09)
    s = slots - shift * bs
    assert np.array_equal(k.double().cpu().numpy(), OQ.values(low[0][s // bs, :, s % bs], low[2][s // bs, :, s % bs]))
    assert np.array_equal(v.double().cpu().numpy(), OQ.values(low[1][s // bs, :, s % bs], low[3][s // bs, :, s % bs]))


# ---------------------------------------------------- graphs, streams, workspaces
def test_captured_calls_follow_their_inputs_and_share_a_workspace():
    """Write and decode captured in two graphs over one workspace, replayed in turn with other
    lengths, tables and tokens."""
    d, bs, Hq, Hkv, B = 128, 16, 8, 2, 3
    lens0 = [2000, 40, 700]
    q, host, tables = decode_case(lens0, d, bs, Hq, Hkv, seed=31, spare=3)
    cache = cache_on_gpu(*[a.copy() for a in host])
    lens_d, tables_d = dev(lens0, torch.int32), dev(tables, torch.int32)
    rng = np.random.default_rng(1)
    kb, vb = (bits(torch.from_numpy(rng.standard_normal((B, Hkv, d))).to(torch.bfloat16)) for _ in range(2))
    k, v = gpu_bf16(kb), gpu_bf16(vb)
    slots_d = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    max_len = tables.shape[1] * bs
    ws = workspace_for(B, Hq, Hkv, d, max_len)
    outs, graphs = [torch.zeros_like(q) for _ in range(2)], []
    for o, scale in zip(outs, (0.1, 0.02)):
        native.paged_attention_decode_quant(q, *cache, tables_d, lens_d, max_len, scale, o, ws)  # warm up
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            native.pkv_write_quant(k, v, slots_d, *cache)
            native.paged_attention_decode_quant(q, *cache, tables_d, lens_d, max_len, scale, o, ws)
        graphs.append(g)
    for lens in ([2000, 40, 700], [1, 0, 31], [1999, 33, 64], [17, 40, 699]):
        slots = np.array([tables[i, (n - 1) // bs] * bs + (n - 1) % bs if n else -1 for i, n in enumerate(lens)])
        slots_d.copy_(dev(slots, torch.int64))
        lens_d.copy_(dev(lens, torch.int32))
        kb, vb = (bits(torch.from_numpy(rng.standard_normal((B, Hkv, d))).to(torch.bfloat16)) for _ in range(2))
        k.copy_(gpu_bf16(kb))
        v.copy_(gpu_bf16(vb))
        OQ.write(kb, vb, slots, *host)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        check_decode(outs[0], q, host, tables, lens, 0.1, f"{lens}")
        check_decode(outs[1], q, host, tables, lens, 0.02, f"{lens}")


def test_two_streams_at_once_with_a_workspace_each():
    lens = [[5000, 3, 1200], [800, 4000, 1]]
    cases = [decode_case(n, 128, 16, 16, 2, seed=40 + i) for i, n in enumerate(lens)]
    caches = [cache_on_gpu(*c[1]) for c in cases]
    ws = [workspace_for(3, 16, 2, 128, 5000) for _ in range(2)]
    outs = [[torch.full_like(c[0], float("nan")) for _ in range(8)] for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(dev(c[2], torch.int32), dev(n, torch.int32)) for c, n in zip(cases, lens)]
    torch.cuda.synchronize()
    for r in range(8):
        for i in range(2):
            native.paged_attention_decode_quant(cases[i][0], *caches[i], *args[i], 5000, 0.1, outs[i][r], ws[i],
                                                stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            check_decode(o, cases[i][0], cases[i][1], cases[i][2], lens[i], 0.1)


def test_back_to_back_calls_over_one_workspace():
    """Steps queued without a wait, as layers of a model: each call's scratch is free for the next."""
    lens = [3000, 64, 900, 2500]
    q, host, tables = decode_case(lens, 64, 32, 8, 2, seed=50)
    cache = cache_on_gpu(*host)
    ws = workspace_for(4, 8, 2, 64, 3000)
    scales = [0.05 * (i + 1) for i in range(12)]
    outs = [torch.full_like(q, float("nan")) for _ in scales]
    t, n = dev(tables, torch.int32), dev(lens, torch.int32)
    torch.cuda.synchronize()
    for o, s in zip(outs, scales):
        native.paged_attention_decode_quant(q, *cache, t, n, 3000, s, o, ws)
    torch.cuda.synchronize()
    for o, s in zip(outs, scales):
        check_decode(o, q, host, tables, lens, s)


@pytest.mark.parametrize("lens,Hq,Hkv", [([30000], 8, 1), ([9000, 7000], 16, 2), ([700, 2300, 1500, 3000, 40, 900], 16, 8)])
def test_a_chain_of_calls_hands_its_data_on(lens, Hq, Hkv):
    """Calls queued without a gap, each reading what the one before wrote (a query from an output, a row
    from a read-back) or a workspace that the one before used: the same bits as one call at a time."""
    d, bs, B = 128, 16, len(lens)
    q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=77)
    cache = cache_on_gpu(*host)
    t, n = dev(tables, torch.int32), dev(lens, torch.int32)
    ws = workspace_for(B, Hq, Hkv, d, max(lens))
    last = dev(np.array([tables[i, (L - 1) // bs] * bs + (L - 1) % bs for i, L in enumerate(lens)]), torch.int64)
    first = dev(np.array([tables[i, 0] * bs for i in range(B)]), torch.int64)
    k, v = (torch.zeros((B, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    a, b = torch.empty_like(q), torch.empty_like(q)

    def chain(wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        c = [x.clone() for x in cache]
        x, outs = q.clone(), []
        torch.cuda.synchronize()
        for i in range(6):
            for src, dst in ((x, a), (a, b), (b, x)):  # every buffer is read, written and read again
                native.paged_attention_decode_quant(src, *c, t, n, max(lens), 0.3, dst, ws)
                pause()
            native.pkv_read_quant(*c, first if i % 2 else last, k, v)
            pause()
            native.pkv_write_quant(k, v, last if i % 2 else first, *c)
            pause()
            if i % 3 == 2:
                outs.append(x.clone())
        torch.cuda.synchronize()
        return outs + [a.clone(), b.clone()] + c

    want = chain(True)
    for _ in range(5):
        for g, w in zip(chain(False), want):
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


# ---------------------------------------------------------- the three together
def as_bf16_blocks(codes, exps):
    """The byte arrays as pkv_block_copy and the swaps take them (include/pkv.h)."""
    NB, Hkv, bs, d = codes.shape
    return codes.view(torch.bfloat16), exps.view(NB, -1).view(torch.bfloat16).view(NB, 1, Hkv * bs // 16, 8)


def test_a_generation_over_the_8_bit_cache():
    """Allocator, prompt write, fork with copy-on-write, token steps, swap out and in, read-back, and
    the bf16 prefill over the read-back rows: each step against the oracle."""
    d, bs, Hq, Hkv = 128, 16, 8, 2
    NB = 64
    rng = np.random.default_rng(77)
    alloc = native.BlockAllocator(NB, bs)
    host = random_cache(NB, Hkv, bs, d, rng, fill=0x7F)
    cache = cache_on_gpu(*[a.copy() for a in host])
    scale = float(np.float32(d ** -0.5))
    st = status_tensor()

    def tokens(n):
        return [bits(torch.from_numpy(rng.standard_normal((n, Hkv, d))).to(torch.bfloat16)) for _ in range(2)]

    def store(slots, kb, vb):
        native.pkv_write_quant(gpu_bf16(kb), gpu_bf16(vb), dev(slots, torch.int64), *cache, st)
        OQ.write(kb, vb, slots, *host)

    for i, n in enumerate((37, 100, 16)):
        alloc.seq_add(i)
        store(alloc.seq_append(i, n), *tokens(n))
    alloc.seq_fork(1, 3)  # shares a partly filled block: the next write copies it
    pair = alloc.seq_cow(3)
    assert pair is not None
    pairs = dev([pair], torch.int32)
    for a, b in ((as_bf16_blocks(cache[0], cache[2])[0], as_bf16_blocks(cache[1], cache[3])[0]),
                 (as_bf16_blocks(cache[0], cache[2])[1], as_bf16_blocks(cache[1], cache[3])[1])):
        native.pkv_block_copy(a, b, pairs, st)
    for a in host:
        a[pair[1]] = a[pair[0]]
    ids = [0, 1, 2, 3]
    for step in range(3):
        store(np.array([alloc.seq_append(i, 1)[0] for i in ids]), *tokens(4))
        tables, lens = alloc.block_table(ids, 10)
        q = torch.from_numpy(rng.standard_normal((4, 1, Hq, d))).to(torch.bfloat16).cuda()
        check_decode(run_decode(q, cache, tables, lens, scale, status=st), q, host, tables, lens, scale, f"step {step}")
    # sequence 1 goes to host memory and comes back in other blocks
    out_ids = alloc.seq_swap_out(1)
    n = len(out_ids)
    hk, hv = (torch.empty((n, Hkv, bs, d // 2), dtype=torch.bfloat16).pin_memory() for _ in range(2))
    hke, hve = (torch.empty((n, 1, Hkv * bs // 16, 8), dtype=torch.bfloat16).pin_memory() for _ in range(2))
    kc, ke = as_bf16_blocks(cache[0], cache[2])
    vc, ve = as_bf16_blocks(cache[1], cache[3])
    native.pkv_swap_out(kc, vc, dev(out_ids, torch.int32), hk, hv, st)
    native.pkv_swap_out(ke, ve, dev(out_ids, torch.int32), hke, hve, st)
    alloc.seq_add(9)
    store(alloc.seq_append(9, 20), *tokens(20))  # takes some of the freed blocks
    in_ids = alloc.seq_swap_in(1)
    native.pkv_swap_in(hk, hv, dev(in_ids, torch.int32), kc, vc, st)
    native.pkv_swap_in(hke, hve, dev(in_ids, torch.int32), ke, ve, st)
    torch.cuda.synchronize()
    tables, lens = alloc.block_table([1], 10)
    # read back through the new slots; the rows are those of the forked sequence up to the fork
    slots = np.array([tables[0, t // bs] * bs + t % bs for t in range(int(lens[0]))])
    k, v = (torch.zeros((len(slots), Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    native.pkv_read_quant(*cache, dev(slots, torch.int64), k, v, st)
    t3, l3 = alloc.block_table([3], 10)
    s3 = np.array([t3[0, t // bs] * bs + t % bs for t in range(100)])
    torch.cuda.synchronize()
    for got, codes, exps in ((k, host[0], host[2]), (v, host[1], host[3])):
        assert np.array_equal(got[:100].double().cpu().numpy(), OQ.values(codes[s3 // bs, :, s3 % bs], exps[s3 // bs, :, s3 % bs]))
    # a prompt chunk's attention over the read-back context in a bf16 cache
    pool = [torch.zeros((10, Hkv, bs, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L = len(slots)
    native.pkv_write(k, v, torch.arange(L, device="cuda"), *pool, st)
    chunk = 5
    q = torch.from_numpy(rng.standard_normal((chunk, Hq, d))).to(torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    native.paged_attention_prefill(q, *pool, torch.arange(10, dtype=torch.int32, device="cuda")[None], dev([L], torch.int32),
                                   dev([0, chunk], torch.int32), scale, out, st)
    torch.cuda.synchronize()
    ref = OA.paged_attention_varlen(bits(q), bits(pool[0]), bits(pool[1]), np.arange(10, dtype=np.int32)[None],
                                    np.array([L], np.int32), np.array([0, chunk], np.int32), num_q_heads=Hq,
                                    num_kv_heads=Hkv, head_dim=d, block_size=bs, scale=scale)
    assert (np.abs(out.double().cpu().numpy() - ref) <= 1e-2 + 1e-2 * np.abs(ref)).all()
    assert st.item() == 0


def test_one_workspace_serves_any_sizes_whatever_it_held():
    """Calls of different sizes in turn over one buffer, which is filled with other bytes before some."""
    cases = [([5000, 40], 128, 16, 16, 2), ([700] * 9, 64, 64, 6, 3), ([33000], 128, 32, 16, 1), ([1, 2, 3], 64, 16, 4, 4)]
    size = max(native.paged_attention_decode_quant_workspace_size(len(n), Hq, Hkv, d, max(n)) for n, d, _, Hq, Hkv in cases)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for round_ in range(3):
        for i, (lens, d, bs, Hq, Hkv) in enumerate(cases):
            if round_ == 1:
                ws.fill_([0, 0xFF, 0xA5, 1][i])
            elif round_ == 2:
                ws.copy_(torch.randint(0, 256, ws.shape, generator=g, device="cuda", dtype=torch.uint8))
            q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=60 + i)
            out = run_decode(q, cache_on_gpu(*host), tables, lens, d ** -0.5, ws=ws)
            check_decode(out, q, host, tables, lens, d ** -0.5, f"round {round_}, case {i}")


@pytest.mark.parametrize("top", [1, 900])
def test_the_largest_batch(top):
    """65535 sequences of no or one token (and three longer ones): a lone value row comes back as it is."""
    B, Hq, Hkv, d, bs = 65535, 2, 1, 64, 16
    rng = np.random.default_rng(top)
    lens = rng.integers(0, 2, B)
    lens[[0, 40000, B - 1]] = top
    host = random_cache(100, Hkv, bs, d, rng)
    tables = rng.integers(0, 100, (B, -(-top // bs))).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((B, 1, Hq, d))).to(torch.bfloat16).cuda()
    out = run_decode(q, cache_on_gpu(*host), tables, lens, 0.125)
    long = np.flatnonzero(lens == top)[:3] if top > 1 else np.array([0])
    check_decode(out[long], q[long], host, tables[long], lens[long], 0.125)
    v = OQ.values(host[1][:, 0, 0], host[3][:, 0, 0])[tables[:, 0]]  # the first token of each sequence's first block
    got = out[:, 0].double().cpu().numpy()
    one = lens == 1
    assert np.array_equal(got[one], np.broadcast_to(v[one][:, None], got[one].shape))
    assert not got[lens == 0].any()


@pytest.mark.parametrize("d,Hq,Hkv,bs,top", [(128, 8, 2, 16, 350), (128, 4, 1, 32, 700), (64, 6, 3, 16, 1500), (128, 32, 2, 64, 256),
                                             (64, 16, 1, 128, 640)])
def test_runs_shared_by_a_ctas_warps_keep_every_piece(d, Hq, Hkv, bs, top):
    """Small batches whose runs are cut over the warps of one CTA, called many times beside a stream that
    keeps the SMs' schedulers busy, so that a CTA's warps start far apart: each warp's piece is joined
    every time (a lost one would leave its tokens out, and no status says so)."""
    rng = np.random.default_rng(top)
    lens = [top, 1] + rng.integers(top // 2, top + 1, 4).tolist()
    q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=top + d)
    assert native.paged_attention_decode_quant_workspace_size(len(lens), Hq, Hkv, d, top) == 0  # no other schedule
    cache = cache_on_gpu(*host)
    t, n = dev(tables, torch.int32), dev(lens, torch.int32)
    want = run_decode(q, cache, tables, lens, d ** -0.5)
    check_decode(want, q, host, tables, lens, d ** -0.5)
    busy, side = torch.randn((1 << 20), device="cuda"), torch.cuda.Stream()
    outs = [torch.full_like(q, float("nan")) for _ in range(300)]
    st = status_tensor()
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        if i % 2 == 0:
            with torch.cuda.stream(side):
                busy.sin_()
        native.paged_attention_decode_quant(q, *cache, t, n, top, d ** -0.5, out, None, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for out in outs:
        assert np.array_equal(bits(out), bits(want))


# ------------------------------------- behind and before the bf16 cache's kernels
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("decodes", ["unsplit", "split", "none listed"])
def test_calls_behind_a_mixed_step_wait_for_its_chunks(decodes, captured):
    """paged_attention_mixed with long chunks beside a few short decodes, which end long before, then at
    once an 8-bit call that reads the chunks' outputs (a decode's queries, a write's rows) or overwrites
    the queries they read (a read-back): the same bits as with a wait in between."""
    Hq, Hkv, bs, d, n_dec, C = 32, 8, 16, 128, 8, 4096
    lens, scale = [60, 200, 1, 17, 33, 128, 90, 150, 8192, 8192], 0.1
    q_start = dev(np.concatenate([np.arange(n_dec + 1), [n_dec + C, n_dec + 2 * C]]), torch.int32)
    rng = np.random.default_rng(3)
    NB = sum(inputs.entries_to_fill(n, bs) for n in lens) + 3
    tables, _ = inputs.permuted_tables(lens, bs, NB, rng, max_blocks=8192 // bs + 2)
    kc, vc = (inputs.randn_bf16((NB, Hkv, bs, d), 90 + i, "cuda") for i in range(2))
    rows = n_dec + 2 * C
    q0 = inputs.randn_bf16((rows, Hq, d), 92, "cuda")
    part = 256 if decodes != "split" else 64
    items = native.pkv_decode_items(np.asarray(lens[:n_dec], dtype=np.int32), tables[:n_dec], Hkv, bs, part, d)
    if decodes == "none listed":
        items = np.zeros_like(items)
    items, t, n = torch.as_tensor(items, device="cuda"), dev(tables, torch.int32), dev(lens, torch.int32)
    ws = torch.empty(max(16, native.paged_attention_workspace_size(n_dec, 1, Hq, d, 200, part)), dtype=torch.uint8,
                     device="cuda")
    # the 8-bit side: a batch of 64 short sequences, whose queries are outputs of the last chunk
    low = [9 + i % 50 for i in range(64)]
    _, host, low_tables = decode_case(low, d, bs, Hq, Hkv, seed=93)
    cache = cache_on_gpu(*host)
    lt, ln = dev(low_tables, torch.int32), dev(low, torch.int32)
    slots = dev([low_tables[i, 0] * bs + i % 9 for i in range(64)], torch.int64)
    many = dev(rng.integers(0, host[0].shape[0] * bs, rows * Hq // Hkv // 2), torch.int64)  # half of q's bytes each
    q, out = q0.clone(), torch.empty_like(q0)
    res = torch.empty((64, 1, Hq, d), dtype=torch.bfloat16, device="cuda")
    st = status_tensor()

    def mixed():
        native.paged_attention_mixed(q, kc, vc, t, n, q_start, scale, out, n_dec, items, 200, part, ws, 100, d_status=st)

    def reads():
        native.paged_attention_decode_quant(out[-64:].unsqueeze(1), *cache, lt, ln, 64, scale, res, None, st)

    def overwrites():
        rows_of_q = q.view(-1, Hkv, d)
        native.pkv_read_quant(*cache, many, rows_of_q[:len(many)], rows_of_q[len(many):], st)

    def writes():
        native.pkv_write_quant(out[-64:, :Hkv], out[-64:, Hkv:2 * Hkv], slots, *cache, st)

    def state():
        return [x.clone() for x in (q, out, res, *cache)]

    def restore(saved):
        for x, s in zip((q, out, res, *cache), saved):
            x.copy_(s)
        torch.cuda.synchronize()

    out.fill_(float("nan"))
    res.fill_(float("nan"))
    start = state()
    for calls in ([overwrites], [reads, overwrites], [writes, reads], [reads, writes, overwrites]):
        restore(start)
        mixed()
        torch.cuda.synchronize()
        for f in calls:
            f()
            torch.cuda.synchronize()
        want = state()
        assert want[1][n_dec:].isfinite().all()
        restore(start)
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                mixed()
                for f in calls:
                    f()
        for _ in range(3):
            restore(start)
            if captured:
                g.replay()
            else:
                mixed()
                for f in calls:
                    f()
            torch.cuda.synchronize()
            for got, w in zip(state(), want):
                assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))
    assert st.item() == 0


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 16, 2), (64, 8, 4)])
def test_a_chain_across_both_caches_hands_its_data_on(d, Hq, Hkv):
    """Calls of the 8-bit and of the bf16 cache queued without a gap, each reading what the one before
    wrote (queries from outputs, cache rows from a read-back) or overwriting what it read: the same
    bits as one call at a time."""
    lens, bs, scale, C = [900, 40, 2500], 16, 0.2, 24
    q, host, tables = decode_case(lens, d, bs, Hq, Hkv, seed=78)
    cache = cache_on_gpu(*host)
    NB, B = host[0].shape[0], len(lens)
    kc, vc = (inputs.randn_bf16((NB, Hkv, bs, d), 95 + i, "cuda") for i in range(2))
    t, n = dev(tables, torch.int32), dev(lens, torch.int32)
    ws8 = workspace_for(B, Hq, Hkv, d, max(lens))
    ws = torch.empty(native.paged_attention_workspace_size(B, 1, Hq, d, max(lens), 256), dtype=torch.uint8, device="cuda")
    last = dev([tables[i, (L - 1) // bs] * bs + (L - 1) % bs for i, L in enumerate(lens)], torch.int64)
    all_slots = dev(np.arange(NB * bs), torch.int64)
    q_start = dev([0, C, 2 * C, 3 * C], torch.int32)
    k, v = (torch.zeros((NB * bs, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    a, b = torch.empty_like(q), torch.empty_like(q)
    chunk, chunk_out = (torch.zeros((3 * C, Hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def chain(wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        c, pool = [x.clone() for x in cache], [kc.clone(), vc.clone()]
        x, rows = q.clone(), inputs.randn_bf16(chunk.shape, 97, "cuda")
        torch.cuda.synchronize()
        for i in range(4):
            native.paged_attention_decode_quant(x, *c, t, n, max(lens), scale, a, ws8)
            pause()
            native.paged_attention_decode(a, *pool, t, n, max(lens), scale, b, ws, 256)
            pause()
            native.paged_attention_decode_quant(b, *c, t, n, max(lens), scale, x, ws8)
            pause()
            native.paged_attention_prefill(rows, *pool, t, n, q_start, scale, chunk_out)
            pause()
            native.pkv_write_quant(chunk_out[:B, :Hkv], chunk_out[C:C + B, :Hkv], last, *c)
            pause()
            native.pkv_read_quant(*c, all_slots, k, v)
            pause()
            # the read-back rows as a bf16 pool of blocks of one head, and as a chunk's queries
            native.paged_attention_prefill(k.view(-1, Hq, d)[:3 * C], *pool, t, n, q_start, scale, rows)
            pause()
            native.pkv_write(k, v, all_slots, *pool)
            pause()
        torch.cuda.synchronize()
        return [a.clone(), b.clone(), x, chunk_out.clone(), rows, k.clone(), v.clone()] + c + pool

    want = chain(True)
    assert all(torch.isfinite(w.float()).all() for w in want[:7])
    for _ in range(4):
        for g, w in zip(chain(False), want):
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_an_overlapped_decode_without_items_wait_for_the_work_ahead(captured):
    """A long prefill, an overlapped list decode whose list names nothing (a graph's bound on an idle
    step), then a read-back over the queries that the prefill reads: the same bits as with waits."""
    Hq, Hkv, bs, d, C = 32, 8, 16, 128, 4096
    NB = 2 * C // bs
    kc, vc, q0 = (inputs.randn_bf16(shape, 99 + i, "cuda") for i, shape in
                  enumerate([(NB, Hkv, bs, d), (NB, Hkv, bs, d), (C, Hq, d)]))
    table, n, q_start = dev([np.arange(NB)], torch.int32), dev([2 * C], torch.int32), dev([0, C], torch.int32)
    dq = inputs.randn_bf16((4, 1, Hq, d), 103, "cuda")
    tables4, lens4 = dev(np.arange(32).reshape(4, 8), torch.int32), dev([40, 1, 128, 77], torch.int32)
    items = torch.zeros((1 + 4 * Hkv, 4), dtype=torch.int32, device="cuda")
    dout = torch.full_like(dq, 3.0)
    host = random_cache(40, Hkv, bs, d, np.random.default_rng(5))
    cache = cache_on_gpu(*host)
    many = dev(np.random.default_rng(6).integers(0, 40 * bs, C * Hq // Hkv // 2), torch.int64)
    q, out, st = q0.clone(), torch.empty_like(q0), status_tensor()

    def run(pause):
        native.paged_attention_prefill(q, kc, vc, table, n, q_start, 0.1, out, st)
        pause()
        native.paged_attention_decode_items(dq, None, None, None, kc, vc, tables4, lens4, 128, 0.1, dout, items,
                                            partition_size=128, d_status=st, overlap=True)
        pause()
        rows = q.view(-1, Hkv, d)
        native.pkv_read_quant(*cache, many, rows[:len(many)], rows[len(many):], st)
        pause()

    def restore():
        q.copy_(q0)
        out.fill_(float("nan"))
        torch.cuda.synchronize()

    restore()
    run(torch.cuda.synchronize)
    want = [q.clone(), out.clone()]
    assert want[1].isfinite().all()
    restore()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(lambda: None)
    for _ in range(4):
        restore()
        if captured:
            g.replay()
        else:
            run(lambda: None)
        torch.cuda.synchronize()
        assert all(np.array_equal(bits(a), bits(b)) for a, b in zip((q, out), want))
    assert (dout == 3.0).all() and st.item() == 0


# how k and v lie: (elements before the first token's rows, tokens' distance less the rows' width)
LIES = {"both 32": ((16, 32), (32, 32)), "k on 16, v on 32": ((8, 32), (0, 32)), "k on 32, v on 16": ((0, 32), (24, 32)),
        "distance of k 8 mod 16": ((0, 24), (16, 32)), "distance of v 8 mod 16": ((16, 32), (0, 40)),
        "k dense, v apart": (None, (16, 48)), "k apart, v dense": ((0, 64), None), "far apart": ((16, 4096), (0, 160))}


@pytest.mark.parametrize("lie", LIES)
@pytest.mark.parametrize("T,Hkv,d", [(301, 2, 64), (40, 3, 48), (130, 8, 128)])
def test_write_of_rows_that_lie_differently(T, Hkv, d, lie):
    """Keys and values in buffers of their own, at other alignments and other distances between tokens:
    32-byte loads where both allow them, 16-byte ones otherwise, bit for bit the same codes."""
    rng = np.random.default_rng(T + d + len(lie))
    bs, width = 16, Hkv * d
    NB = -(-T // bs) + 2
    slots = inputs.distinct_slots(T, NB * bs, rng, skip_fraction=0.1)
    host = random_cache(NB, Hkv, bs, d, rng, fill=0xAB)
    cache = cache_on_gpu(*[a.copy() for a in host])
    rows = [awkward_rows(T, Hkv, d, rng) for _ in range(2)]
    placed = []
    for b, where in zip(rows, LIES[lie]):
        if where is None:
            placed.append(gpu_bf16(b))
            continue
        start, more = where
        buf = torch.full((start + T * (width + more),), float("nan"), dtype=torch.bfloat16, device="cuda")
        assert buf.data_ptr() % 32 == 0
        t = buf[start:].view(T, width + more)[:, :width].view(T, Hkv, d)
        t.copy_(gpu_bf16(b))
        assert t.stride(0) == width + more and t.data_ptr() % 32 == (16 if start % 16 else 0)
        placed.append(t)
    OQ.write(*rows, slots, *host)
    st = status_tensor()
    native.pkv_write_quant(*placed, dev(slots, torch.int64), *cache, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert all(np.array_equal(u8(got), want) for got, want in zip(cache, host))
