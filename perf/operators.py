"""Performance cases of the 8-bit KV cache: its write, its read-back and the
single-token decode over it, each with a plain form in elementary torch
operations.

The cache: per (token, KV head) a key row and a value row of e4m3 codes and, for
each row, one exponent byte b; a code c stands for c * 2^(b - 127).  Laid out in
blocks like the bf16 cache: codes [blocks][KV heads][block size][head dim],
exponents [blocks][KV heads][block size].

``own`` chooses between the plain forms (False) and the library's calls (True).
"""
import math

import numpy as np
import torch

own = False

_E_MIN, _E_MAX, _BIAS, _TOP = -31, 31, 127, 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest decode: three short sequences, four query heads (latency only)
        _decode("decode_tiny", batch=3, q_heads=4, kv_heads=2, head_dim=64, block=16, length=64, spread="uniform"),
        # one user with a long context: few rows, a long axis to split
        _decode("decode_one_long", batch=1, q_heads=64, kv_heads=8, head_dim=128, block=16, length=32768,
                spread="equal"),
        # a batch of chats of all ages
        _decode("decode_batch", batch=32, q_heads=32, kv_heads=8, head_dim=128, block=16, length=4096,
                spread="uniform"),
        # a continuous-batching step: many short sequences, a few long ones
        _decode("decode_mix", batch=256, q_heads=32, kv_heads=8, head_dim=128, block=16, length=8192,
                spread="lognormal"),
        # long contexts throughout, the largest decode
        _decode("decode_long", batch=16, q_heads=64, kv_heads=8, head_dim=128, block=32, length=32768,
                spread="equal"),
        # one KV head per query head, narrow heads, odd lengths, large blocks
        _decode("decode_no_groups", batch=61, q_heads=16, kv_heads=16, head_dim=64, block=64, length=2047,
                spread="uniform"),
        # sixteen query heads share a KV head; the longest block
        _decode("decode_wide_group", batch=48, q_heads=32, kv_heads=2, head_dim=128, block=128, length=9001,
                spread="uniform"),
        # the new tokens of one decode step, some of them already cached (skipped)
        _rows("write_step", "write", tokens=256, kv_heads=8, head_dim=128, block=16, skip=0.1, strided=False),
        # a prompt's chunk, its rows taken as views of a fused projection's output
        _rows("write_chunk", "write", tokens=8192, kv_heads=8, head_dim=128, block=16, skip=0.0, strided=True),
        # whole prompts in one call, the largest write
        _rows("write_prompts", "write", tokens=32768, kv_heads=8, head_dim=128, block=16, skip=0.0, strided=False),
        # a short stretch read back (a prefix compared or handed on)
        _rows("read_stretch", "read", tokens=1021, kv_heads=2, head_dim=64, block=32, skip=0.1, strided=False),
        # a whole long context read back into bf16 for a prompt chunk's attention
        _rows("read_context", "read", tokens=32768, kv_heads=8, head_dim=128, block=16, skip=0.0, strided=False),
    ]


def _decode(name, **c):
    return {"name": name, "op": "decode", **c}


def _rows(name, op, **c):
    return {"name": name, "op": op, **c}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        head_dim = rng.choice((64, 128))
        kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
        batch = _log_int(rng, 1, 512)
        room = 16 * 32768 * 8 * 128 // (batch * kv_heads * head_dim * max(1, group // 8))
        return {"op": "decode", "batch": batch, "q_heads": kv_heads * group, "kv_heads": kv_heads,
                "head_dim": head_dim, "block": rng.choice((16, 32, 64, 128)),
                "length": _log_int(rng, 1, max(1, min(65536, room))),
                "spread": rng.choice(("equal", "uniform", "lognormal"))}
    head_dim = rng.choice((16, 48, 64, 80, 96, 112, 128, 192, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
    room = 32768 * 8 * 128 // (kv_heads * head_dim)
    op = rng.choice(("write", "read"))
    return {"op": op, "tokens": _log_int(rng, 1, min(65536, room)), "kv_heads": kv_heads, "head_dim": head_dim,
            "block": rng.choice((1, 8, 16, 24, 32, 64, 128)), "skip": rng.choice((0.0, 0.1)),
            "strided": op == "write" and rng.random() < 0.5}


def _lengths(case):
    """The decode's sequence lengths: a function of the case alone."""
    rng = np.random.default_rng([case["batch"], case["length"], case["q_heads"]])
    top, n = case["length"], case["batch"]
    if case["spread"] == "equal":
        return np.full(n, top, dtype=np.int64)
    if case["spread"] == "uniform":
        return rng.integers(1, top + 1, size=n)
    x = np.exp(np.log(max(1.0, top / 16)) + rng.standard_normal(n))
    return np.clip(np.rint(x), 1, top).astype(np.int64)


def work(case):
    hkv, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "decode":
        lens = _lengths(case)
        keys = int(lens.sum())
        blocks = int((-(-lens // case["block"])).sum())
        rows = case["batch"] * case["q_heads"]
        return {"bytes": keys * hkv * 2 * (d + 1) + 4 * blocks + 4 * case["batch"] + 2 * 2 * rows * d,
                "flops": 4 * case["q_heads"] * d * keys}
    moved = case["tokens"] - _skipped(case)
    return {"bytes": moved * hkv * 2 * (3 * d + 1) + 8 * case["tokens"], "flops": 2 * moved * hkv * 2 * d}


def _skipped(case):
    return int(case["tokens"] * case["skip"])


# ----------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _power(e):
    """2^e in fp32 for an integer tensor e in [-126, 127], exactly (the exponent field)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of x (fp32) -> (e4m3 codes, exponent bytes)."""
    finite = torch.isfinite(x)
    a = torch.where(finite, x.abs(), 0.0).amax(-1)
    m, p = torch.frexp(a)  # a = m 2^p, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(a > 0, p - 9 + (m > 0.875), _E_MIN).clamp(_E_MIN, _E_MAX)
    y = (x * _power(-e)[..., None]).clamp(-_TOP, _TOP)
    codes = torch.where(finite, y, float("nan")).to(torch.float8_e4m3fn)
    return codes, (e + _BIAS).to(torch.uint8)


def _rows_like(shape, g, channels):
    """Rows as a model's projections give them: N(0, 1) times a size per channel."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * channels).to(torch.bfloat16)


def _channels(d, g, outliers):
    """Channel sizes: a spread around 1 and, for keys, a few channels many times larger."""
    c = torch.exp(0.3 * torch.randn(d, generator=g, device="cuda"))
    if outliers:
        c[torch.randint(0, d, (max(1, d // 32),), generator=g, device="cuda")] *= 8.0
    return c


def _filled_cache(blocks, hkv, bs, d, g):
    """A cache that holds tokens throughout: codes and exponents of keys and of values."""
    out = []
    for outliers in (True, False):
        ch = _channels(d, g, outliers)
        codes = torch.empty((blocks, hkv, bs, d), dtype=torch.uint8, device="cuda")
        exps = torch.empty((blocks, hkv, bs), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (hkv * bs * d))
        for b in range(0, blocks, step):
            n = min(step, blocks - b)
            c, e = _quantise(_rows_like((n, hkv, bs, d), g, ch).float())
            codes[b:b + n] = c.view(torch.uint8)
            exps[b:b + n] = e
        out.append((codes.view(torch.float8_e4m3fn), exps))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def prepare(case, seed):
    g = _generator(seed * 1000003 + 17)
    hkv, d, bs = case["kv_heads"], case["head_dim"], case["block"]
    rng = np.random.default_rng([int(seed), hkv, d, bs])
    state = {"op": case["op"], "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "decode":
        lens = _lengths(case)
        counts = -(-lens // bs)
        blocks = int(counts.sum()) + 3
        perm = rng.permutation(blocks)
        tables = np.full((len(lens), int(counts.max())), -1, dtype=np.int32)
        at = 0
        for i, c in enumerate(counts):
            tables[i, :c] = perm[at:at + c]
            at += c
        state["cache"] = _filled_cache(blocks, hkv, bs, d, g)
        state["q"] = _rows_like((len(lens), 1, case["q_heads"], d), g, _channels(d, g, False))
        state["tables"] = torch.as_tensor(tables, device="cuda")
        state["lens"] = torch.as_tensor(lens.astype(np.int32), device="cuda")
        state["max_len"] = int(lens.max())
        state["scale"] = float(np.float32(d ** -0.5))
        state["out"] = torch.zeros_like(state["q"])
        state["workspace"] = None
        return state
    tokens = case["tokens"]
    blocks = -(-tokens // bs) + 2
    # a block more than the pool, for the plain form's skipped rows
    cache = _filled_cache(blocks + 1, hkv, bs, d, g)
    state["spare"] = cache
    state["cache"] = tuple(t[:blocks] for t in cache)
    order = rng.permutation(blocks)[:-(-tokens // bs)]  # whole blocks in random order, as an allocator hands them out
    slots = (order[:, None] * bs + np.arange(bs)[None, :]).reshape(-1)[:tokens].astype(np.int64)
    slots[rng.permutation(tokens)[:_skipped(case)]] = -1
    state["slots"] = torch.as_tensor(slots, device="cuda")
    if case["op"] == "write":
        kc, vc = _channels(d, g, True), _channels(d, g, False)
        if case["strided"]:  # [token][query heads | key heads | value heads], two query heads per KV head
            fused = torch.empty((tokens, 4 * hkv, d), dtype=torch.bfloat16, device="cuda")
            fused[:, 2 * hkv:3 * hkv] = _rows_like((tokens, hkv, d), g, kc)
            fused[:, 3 * hkv:] = _rows_like((tokens, hkv, d), g, vc)
            fused[:, :2 * hkv] = 0.0
            state["k"], state["v"] = fused[:, 2 * hkv:3 * hkv], fused[:, 3 * hkv:]
        else:
            state["k"], state["v"] = _rows_like((tokens, hkv, d), g, kc), _rows_like((tokens, hkv, d), g, vc)
    else:
        state["k"] = torch.zeros((tokens, hkv, d), dtype=torch.bfloat16, device="cuda")
        state["v"] = torch.zeros_like(state["k"])
    return state


# -------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return {"decode": _plain_decode, "write": _plain_write, "read": _plain_read}[state["op"]](state)


def _run_own(s):
    from paged_kv_cache_276_gb300 import native
    if s["op"] == "decode":
        if s["workspace"] is None:  # once, as a program keeps it
            b, _, hq, d = s["q"].shape
            n = native.paged_attention_decode_quant_workspace_size(b, hq, s["cache"][0].shape[1], d, s["max_len"])
            s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        native.paged_attention_decode_quant(s["q"], *s["cache"], s["tables"], s["lens"], s["max_len"], s["scale"],
                                            s["out"], s["workspace"], s["status"])
        return s["out"]
    if s["op"] == "write":
        native.pkv_write_quant(s["k"], s["v"], s["slots"], *s["cache"], s["status"])
        return s["cache"]
    native.pkv_read_quant(*s["cache"], s["slots"], s["k"], s["v"], s["status"])
    return s["k"], s["v"]


def _values(codes, exps):
    return codes.view(torch.float8_e4m3fn).float() * _power(exps.to(torch.int32) - _BIAS)[..., None]


def _plain_decode(s):
    kc, vc, ke, ve = s["cache"]
    b, _, hq, d = s["q"].shape
    hkv, bs = kc.shape[1], kc.shape[2]
    ids = s["tables"].clamp(min=0).long()

    def gather(codes, exps):  # [B, blocks, Hkv, bs, d] -> [B, Hkv, tokens, d]
        x = _values(codes.view(torch.uint8)[ids], exps[ids])
        return x.permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)

    k = gather(kc, ke)
    q = s["q"].float().reshape(b, hkv, hq // hkv, d)
    scores = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    seen = torch.arange(scores.shape[-1], device="cuda")[None, :] < s["lens"][:, None]  # [B, tokens]
    scores = scores.masked_fill(~seen[:, None, None, :], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(top > float("-inf"), top, 0.0))
    total = w.sum(-1, keepdim=True)
    v = gather(vc, ve).masked_fill(~seen[:, None, :, None], 0.0)
    o = torch.matmul(w, v) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.reshape(b, 1, hq, d))
    return s["out"]


def _plain_write(s):
    hkv, bs = s["cache"][0].shape[1], s["cache"][0].shape[2]
    blocks = s["cache"][0].shape[0]
    slots = torch.where(s["slots"] >= 0, s["slots"], blocks * bs)  # skipped rows land in the block past the pool
    at, off = slots // bs, slots % bs
    for x, codes, exps in ((s["k"], s["spare"][0], s["spare"][2]), (s["v"], s["spare"][1], s["spare"][3])):
        c, e = _quantise(x.float())
        codes.view(torch.uint8)[at, :, off] = c.view(torch.uint8)
        exps[at, :, off] = e
    return s["cache"]


def _plain_read(s):
    bs = s["cache"][0].shape[2]
    keep = (s["slots"] >= 0)[:, None, None]
    slots = s["slots"].clamp(min=0)
    at, off = slots // bs, slots % bs
    kc, vc, ke, ve = s["cache"]
    for out, codes, exps in ((s["k"], kc, ke), (s["v"], vc, ve)):
        out.copy_(torch.where(keep, _values(codes.view(torch.uint8)[at, :, off], exps[at, :, off]), out.float()))
    return s["k"], s["v"]


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definition in 64 bits, sequence by sequence and row by row."""
    s = prepare(case, seed)
    kc, vc, ke, ve = (t.clone() for t in s["cache"])
    if case["op"] == "decode":
        b, _, hq, d = s["q"].shape
        hkv = kc.shape[1]
        out = torch.zeros((b, 1, hq, d), dtype=torch.float64, device="cuda")
        for i, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            ids = s["tables"][i, :-(-n // case["block"])].long()

            def whole(codes, exps):
                x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(torch.float64)
                x = x * torch.exp2(exps[ids].to(torch.float64) - 127.0)[..., None]
                return x.transpose(0, 1).reshape(hkv, -1, d)[:, :n]

            q = s["q"][i, 0].double().reshape(hkv, hq // hkv, d)
            z = torch.einsum("hgd,htd->hgt", q, whole(kc, ke)) * s["scale"]
            out[i, 0] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), whole(vc, ve)).reshape(hq, d)
        return out
    bs = case["block"]
    slots = s["slots"]
    live = (slots >= 0).nonzero()[:, 0]
    at, off = slots[live] // bs, slots[live] % bs
    if case["op"] == "read":
        got = []
        for codes, exps in ((kc, ke), (vc, ve)):
            x = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
            c = codes.view(torch.uint8)[at, :, off].view(torch.float8_e4m3fn).to(torch.float64)
            x[live] = c * torch.exp2(exps[at, :, off].to(torch.float64) - 127.0)[..., None]
            got.append(x)
        return tuple(got)
    got = []
    for x, codes in ((s["k"], kc), (s["v"], vc)):
        y = codes.to(torch.float64)
        r = x[live].to(torch.float64)
        a = r.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -300) / 448.0) - 1e-12).clamp(-31, 31)
        y[at, :, off] = r * torch.exp2(-e)  # what the codes round
        got.append(y)
    return got[0], got[1], None, None
