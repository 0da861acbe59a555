"""Oracle of the 8-bit cache: rows of e4m3 codes with a power-of-two exponent
byte, in float64 numpy, one value at a time in meaning (vectorised in form).

e4m3: 1 sign bit, 4 exponent bits (bias 7), 3 mantissa bits, no infinities,
NaN = all other bits set, largest finite value 448, smallest step 2^-9.
"""
import numpy as np

E_MIN, E_MAX, BIAS, TOP = -31, 31, 127, 448.0


def bf16_values(bits):
    """bf16 bit patterns (uint16) -> float64."""
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_bits(x):
    """float64 values that bf16 holds exactly (or NaN) -> bit patterns."""
    b = np.asarray(x, dtype=np.float64).astype(np.float32).view(np.uint32)
    assert ((b & 0xFFFF) == 0)[np.isfinite(x)].all(), "not a bf16 value"
    return (b >> 16).astype(np.uint16)


def code_table():
    """The values of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** -9
        else:
            out[c] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


TABLE = code_table()


def encode(y):
    """float64 -> codes: nearest, ties to even, held at +-448; NaN -> 0x7F."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), TOP)
    a = np.where(np.isnan(y), 0.0, a)
    _, p = np.frexp(a)  # a = m 2^p, m in [0.5, 1): floor(log2 a) = p - 1
    step = 2.0 ** (np.maximum(p - 1, -6) - 3)
    n = np.rint(a / step) * step  # rint: half to even
    _, p = np.frexp(n)
    ex = p - 1
    normal = n >= 2.0 ** -6
    code = np.where(normal, ((ex + 7) << 3) + np.rint((n / 2.0 ** ex - 1) * 8 * normal).astype(np.int64),
                    np.rint(n * 2.0 ** 9 * ~normal).astype(np.int64))
    code = code | np.where(np.signbit(y), 0x80, 0)
    return np.where(np.isnan(y), 0x7F, code).astype(np.uint8)


def row_exponents(x):
    """[..., d] float64 rows -> the smallest e with max |finite x| <= 448 * 2^e, clamped (int)."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    too_small = TOP * 2.0 ** np.arange(E_MIN, E_MAX, dtype=np.float64)  # 448 * 2^k: e is above k where it is below a
    return E_MIN + np.searchsorted(too_small, a, side="left")


def quantise(bits):
    """[..., d] bf16 bit patterns -> (codes [..., d], exponent bytes [...])."""
    x = bf16_values(bits)
    e = row_exponents(x)
    y = np.where(np.isfinite(x), x, np.nan) * 2.0 ** -e.astype(np.float64)[..., None]
    return encode(y), (e + BIAS).astype(np.uint8)


def values(codes, exps):
    """What stored rows stand for, float64 (exponent bytes no write stores count as the nearer bound)."""
    e = np.clip(np.asarray(exps).astype(np.int64), E_MIN + BIAS, E_MAX + BIAS) - BIAS
    return TABLE[codes] * 2.0 ** e.astype(np.float64)[..., None]


def write(k_bits, v_bits, slots, k_codes, v_codes, k_exps, v_exps):
    """In place: quantised rows of token t to slot slots[t] (negative: none)."""
    bs = k_codes.shape[2]
    for t, s in enumerate(np.asarray(slots).tolist()):
        if s < 0:
            continue
        b, o = divmod(s, bs)
        for bits, codes, exps in ((k_bits, k_codes, k_exps), (v_bits, v_codes, v_exps)):
            codes[b, :, o], exps[b, :, o] = quantise(bits[t])


def decode(q_bits, k_codes, v_codes, k_exps, v_exps, tables, lens, scale):
    """fp64 attention of one token per sequence.  q [B, Hq, d] bf16 bits.  Returns
    (out [B, Hq, d], and for error bounds: sum_t p_t |v_t| [B, Hq, d], the largest
    scale * sum_i |q_i k_ti| [B, Hq], and the largest p_t 2^ve_t [B, Hq])."""
    q = bf16_values(q_bits)
    B, Hq, d = q.shape
    Hkv, bs = k_codes.shape[1], k_codes.shape[2]
    G = Hq // Hkv
    out, mag = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    dot, top = np.zeros((B, Hq)), np.zeros((B, Hq))
    for i in range(B):
        L = int(lens[i])
        if L == 0:
            continue
        ids = np.array([int(tables[i][j]) for j in range(-(-L // bs))])

        def rows(x):  # the sequence's blocks in order, one KV head after the other: [Hkv, L, ...]
            x = x[ids].swapaxes(0, 1)
            return x.reshape((Hkv, len(ids) * bs) + x.shape[3:])[:, :L]

        k, v = values(rows(k_codes), rows(k_exps)), values(rows(v_codes), rows(v_exps))
        ve = np.clip(rows(v_exps).astype(np.int64), E_MIN + BIAS, E_MAX + BIAS) - BIAS
        qi = q[i].reshape(Hkv, G, d)  # query head g reads KV head g // G
        s = (qi @ k.swapaxes(1, 2)) * scale
        w = np.exp(s - s.max(-1, keepdims=True))
        w = w / w.sum(-1, keepdims=True)
        out[i] = (w @ v).reshape(Hq, d)
        mag[i] = (w @ np.abs(v)).reshape(Hq, d)
        dot[i] = (np.abs(qi) @ np.abs(k).swapaxes(1, 2)).max(-1).reshape(Hq) * abs(scale)
        top[i] = (w * 2.0 ** ve.astype(np.float64)[:, None, :]).max(-1).reshape(Hq)
    return out, mag, dot, top
