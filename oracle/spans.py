"""Oracle of windowed and tree attention: float64, every row over the keys it sees,
gathered from the blocks one sequence at a time."""
import numpy as np

from .quant import bf16_values


def window_sees(L, c, window, sinks):
    """[c, L]: row r at position p = L - c + r sees t <= p with t > p - window or t < sinks."""
    p, t = np.arange(L - c, L)[:, None], np.arange(L)[None]
    return (t <= p) & ((t > p - window) | (t < sinks))


def tree_sees(L, c, words):
    """[c, L]: every t < L - c, and t = L - c + j where bit j of the row's word is set."""
    out = np.zeros((c, L), dtype=bool)
    for r in range(c):
        for t in range(L):
            j = t - (L - c)
            out[r, t] = j < 0 or bool((int(words[r]) >> j) & 1)
    return out


def attend(q_bits, k_bits, v_bits, tables, lens, q_start, scale, sees):
    """q [total_q, Hq, d], caches [NB, Hkv, bs, d] (bf16 bits); sees: per sequence a bool [c, L].  Returns
    (out [total_q, Hq, d], sum_t p_t |v_t| of the same shape, and per row and head the largest
    scale * sum_i |q_i k_ti| over the keys seen).  Rows that see nothing: zeros."""
    q = bf16_values(q_bits)
    n, hq, d = q.shape
    hkv, bs = k_bits.shape[1], k_bits.shape[2]
    out, mag, dot = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq))
    for i, L in enumerate(lens):
        a, e = int(q_start[i]), int(q_start[i + 1])
        cols = np.nonzero(sees[i].any(0))[0] if sees[i].size else np.zeros(0, dtype=int)
        if not len(cols):
            continue
        blocks = np.array([int(tables[i][t // bs]) for t in cols])
        k, v = (bf16_values(x[blocks, :, cols % bs]).swapaxes(0, 1) for x in (k_bits, v_bits))  # [Hkv, n, d]
        seen = sees[i][:, cols]
        qi = q[a:e].reshape(e - a, hkv, hq // hkv, d).transpose(1, 2, 0, 3)  # [Hkv, G, c, d]
        with np.errstate(invalid="ignore", over="ignore"):
            s = np.where(seen, qi @ k[:, None].swapaxes(-1, -2) * scale, -np.inf)
            top = s.max(-1, keepdims=True)
            w = np.where(seen, np.exp(s - np.where(top > -np.inf, top, 0.0)), 0.0)
            total = w.sum(-1, keepdims=True)
            w = w / np.where(total == 0, 1.0, total)

            def rows(x):  # [Hkv, G, c, ...] -> [c, Hq, ...]
                return np.moveaxis(x, 2, 0).reshape((e - a, hq) + x.shape[3:])

            if np.isfinite(v).all():
                o, m = w @ v[:, None], w @ np.abs(v)[:, None]
            else:  # a value that is not seen takes no part, whatever it is
                o, m = np.zeros(qi.shape), np.zeros(qi.shape)
                for r in range(e - a):
                    z = np.nonzero(seen[r])[0]
                    wr, vr = w[:, :, r:r + 1][..., z], v[:, z][:, None]
                    o[:, :, r], m[:, :, r] = (wr @ vr)[:, :, 0], (wr @ np.abs(vr))[:, :, 0]
            out[a:e], mag[a:e] = rows(o), rows(m)
            ka = np.where(np.isfinite(k), np.abs(k), 0.0)
            g = np.where(seen, np.abs(qi) @ ka[:, None].swapaxes(-1, -2), 0.0).max(-1) * abs(scale)
            dot[a:e] = rows(g)
    return out, mag, dot
