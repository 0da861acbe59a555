"""Performance cases of three operators over the paged bf16 and 8-bit caches, each
with a plain form in elementary torch operations:

* the rotary append: queries and keys rotated to their positions, the queries
  written out, keys and values stored into their cache slots (bf16 or 8-bit);
* attention of a tree of drafted tokens over the cache: every node sees the
  whole context and, by a 64-bit mask, some of its tree;
* attention with a sliding window and a few first tokens that stay visible, for
  single tokens and for prompt chunks.

``own`` chooses between the plain forms (False) and the library's calls (True).
"""
import math

import numpy as np
import torch

own = False

_E_MIN, _E_MAX, _BIAS, _TOP = -31, 31, 127, 448.0  # the 8-bit cache's exponents and largest code


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the new tokens of one decode step, some of them already cached (not stored)
        _rope("rope_step", tokens=256, q_heads=32, kv_heads=8, head_dim=128, rot=128, style="half", block=16,
              cache="bf16", skip=0.1, strided=False, positions=8192),
        # whole prompts in one call out of a fused projection, the largest append
        _rope("rope_prompts", tokens=32768, q_heads=32, kv_heads=8, head_dim=128, rot=128, style="half", block=16,
              cache="bf16", skip=0.0, strided=True, positions=32768),
        # a stretch of odd length, half of narrow heads rotated, as many KV heads as query heads
        _rope("rope_partial", tokens=1021, q_heads=16, kv_heads=16, head_dim=64, rot=32, style="pairs", block=64,
              cache="bf16", skip=0.1, strided=True, positions=131072),
        # a prompt's chunk into the 8-bit cache
        _rope("rope_chunk_8bit", tokens=8192, q_heads=64, kv_heads=8, head_dim=128, rot=128, style="pairs", block=32,
              cache="8bit", skip=0.0, strided=True, positions=32768),
        # the smallest trees: three short sequences (latency only)
        _tree("tree_tiny", batch=3, nodes=8, q_heads=4, kv_heads=2, head_dim=64, block=16, length=64,
              spread="uniform"),
        # one user with a long context and the widest tree: few rows, a long axis to split
        _tree("tree_one_long", batch=1, nodes=64, q_heads=64, kv_heads=8, head_dim=128, block=16, length=32768,
              spread="equal"),
        # a batch of chats of all ages, trees of up to 26 nodes
        _tree("tree_batch", batch=32, nodes=26, q_heads=32, kv_heads=8, head_dim=128, block=16, length=4096,
              spread="uniform"),
        # a continuous-batching step with short drafts: many short sequences, a few long ones
        _tree("tree_mix", batch=256, nodes=8, q_heads=32, kv_heads=8, head_dim=128, block=16, length=8192,
              spread="lognormal"),
        # a continuous-batching decode step of a windowed layer
        _window("window_step", batch=256, chunk=1, q_heads=32, kv_heads=8, head_dim=128, block=16, length=8192,
                spread="lognormal", window=1024, sinks=4),
        # long contexts behind a wide window, single tokens
        _window("window_long", batch=16, chunk=1, q_heads=64, kv_heads=8, head_dim=128, block=32, length=32768,
                spread="equal", window=4096, sinks=16),
        # whole prompts through a windowed layer, the largest
        _window("window_prompts", batch=4, chunk=8192, q_heads=32, kv_heads=8, head_dim=128, block=16, length=8192,
                spread="equal", window=1024, sinks=4),
        # ragged chunks behind contexts of all lengths, narrow heads without groups, an odd window, no sinks
        _window("window_chunks", batch=9, chunk=517, q_heads=16, kv_heads=16, head_dim=64, block=64, length=16384,
                spread="uniform", window=2047, sinks=0),
    ]


def _rope(name, **c):
    return {"name": name, "op": "rope", **c}


def _tree(name, **c):
    return {"name": name, "op": "tree", **c}


def _window(name, **c):
    return {"name": name, "op": "window", **c}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_ROPE_ROOM = 32768 * 48 * 128    # values of the largest append
_KEY_ROOM = 16 * 32768 * 8 * 128  # key values that a call's sequences hold at most
_SCORE_ROOM = 1 << 29            # scores of a call


def draw(rng):
    op = rng.choice(("rope", "tree", "window"))
    if op == "rope":
        head_dim = rng.choice((16, 48, 64, 80, 96, 112, 128, 192, 256))
        kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
        group = rng.choice((1, 2, 3, 4, 7, 8, 16))
        room = _ROPE_ROOM // ((group + 2) * kv_heads * head_dim)
        return {"op": op, "tokens": _log_int(rng, 1, min(65536, room)), "q_heads": kv_heads * group,
                "kv_heads": kv_heads, "head_dim": head_dim, "rot": 16 * rng.randint(1, head_dim // 16),
                "style": rng.choice(("half", "pairs")), "block": rng.choice((1, 8, 16, 24, 32, 64, 128)),
                "cache": rng.choice(("bf16", "8bit")), "skip": rng.choice((0.0, 0.1)),
                "strided": rng.random() < 0.5, "positions": rng.choice((4096, 32768, 131072))}
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
    batch = _log_int(rng, 1, 256)
    case = {"op": op, "batch": batch, "q_heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim,
            "block": rng.choice((16, 32, 64, 128)), "spread": rng.choice(("equal", "uniform", "lognormal"))}
    keys = _KEY_ROOM // (batch * kv_heads * head_dim)
    if op == "tree":
        case["nodes"] = _log_int(rng, 1, 64)
        keys = min(keys, _SCORE_ROOM // (batch * case["q_heads"] * case["nodes"]), 65536)
        case["length"] = _log_int(rng, min(case["nodes"], keys), max(case["nodes"], keys))
        return case
    case["window"] = _log_int(rng, 1, 8192)
    case["sinks"] = rng.choice((0, 0, 1, 4, 16, 130))
    if rng.random() < 0.5:
        case["chunk"] = 1
        case["length"] = _log_int(rng, 1, max(1, min(65536, keys)))
        return case
    case["chunk"] = _log_int(rng, 2, max(2, min(8192, 32768 // batch)))
    seen = case["window"] + case["sinks"] + 1024  # keys of one stretch of queries
    rows = max(2, _SCORE_ROOM * 2 // (seen * batch * case["q_heads"]))
    case["chunk"] = min(case["chunk"], rows)
    case["length"] = _log_int(rng, case["chunk"], max(case["chunk"], min(65536, keys)))
    return case


def _lengths(case):
    """Every sequence's tokens, its newest ones included: a function of the case alone."""
    rng = np.random.default_rng([case["batch"], case["length"], case["q_heads"]])
    top, n = case["length"], case["batch"]
    if case["spread"] == "equal":
        return np.full(n, top, dtype=np.int64)
    if case["spread"] == "uniform":
        return rng.integers(1, top + 1, size=n)
    x = np.exp(np.log(max(1.0, top / 16)) + rng.standard_normal(n))
    return np.clip(np.rint(x), 1, top).astype(np.int64)


def _rows(case):
    """Every sequence's query tokens: all of the chunk or tree, or (mixed lengths) fewer."""
    lens = _lengths(case)
    top = case["nodes"] if case["op"] == "tree" else case["chunk"]
    if case["spread"] == "equal" or top == 1:
        return np.minimum(top, lens)
    rng = np.random.default_rng([case["batch"], top, 7])
    return np.minimum(lens, rng.integers(max(1, top // 2), top + 1, size=case["batch"]))


def _skipped(case):
    return int(case["tokens"] * case["skip"])


def work(case):
    hkv, hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    if case["op"] == "rope":
        n, kept = case["tokens"], case["tokens"] - _skipped(case)
        stored = 2 * (d + 1) if case["cache"] == "8bit" else 4 * d
        table = 4 * case["rot"] * min(n, case["positions"])
        return {"bytes": n * hq * 4 * d + kept * hkv * (4 * d + stored) + 16 * n + table,
                "flops": 3 * case["rot"] * (n * hq + kept * hkv)}
    lens, rows = _lengths(case), _rows(case)
    ctx = lens - rows
    if case["op"] == "tree":
        read = lens
        pairs = (rows * lens).sum()  # (query token, key): the nodes' own part is small
        extra = 8 * rows.sum()
    else:
        w, s = case["window"], case["sinks"]
        first = np.maximum(0, ctx - w + 1)
        read = lens - np.maximum(0, first - s)
        # token p sees min(p + 1, w) of its window and the sinks before it
        pairs = 0
        for a, b in zip(ctx, lens):
            p = np.arange(a, b)
            pairs += int((np.minimum(p + 1, w) + np.minimum(s, np.maximum(0, p + 1 - w))).sum())
        extra = 0
    blocks = int((-(-read // case["block"])).sum())
    return {"bytes": int(read.sum()) * hkv * 4 * d + 4 * blocks + 8 * case["batch"] + 4 * int(rows.sum()) * hq * d
            + int(extra), "flops": 4 * hq * d * int(pairs)}


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


def _channels(d, g, outliers):
    """Channel sizes: a spread around 1 and, for keys, a few channels many times larger."""
    c = torch.exp(0.3 * torch.randn(d, generator=g, device="cuda"))
    if outliers:
        c[torch.randint(0, d, (max(1, d // 32),), generator=g, device="cuda")] *= 8.0
    return c


def _rows_like(shape, g, channels):
    """Rows as a model's projections give them: N(0, 1) times a size per channel."""
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * channels).to(torch.bfloat16)


def _table(positions, rot):
    """[positions, rot]: the cosines of the rot / 2 angles of each position, then their sines."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _tree_masks(rows, rng):
    """A random tree per sequence (every node's parent comes before it): each node's ancestors and itself, as bits."""
    out = []
    for n in rows:
        m = []
        for j in range(n):
            parent = int(rng.integers(-1, j)) if j else -1
            m.append((m[parent] if parent >= 0 else 0) | (1 << j))
        out += m
    return np.array(out, dtype=np.uint64).view(np.int64)


def prepare(case, seed):
    g = _generator(seed * 1000003 + 29)
    hq, hkv, d, bs = case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    rng = np.random.default_rng([int(seed), hkv, d, bs])
    state = {"op": case["op"], "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    return (_prepare_rope if case["op"] == "rope" else _prepare_attention)(case, state, g, rng, hq, hkv, d, bs)


def _prepare_rope(case, state, g, rng, hq, hkv, d, bs):
    n, top = case["tokens"], case["positions"]
    blocks = -(-n // bs) + 2
    # a block more than the pool, for the plain form's skipped rows
    shape = (blocks + 1, hkv, bs)
    if case["cache"] == "8bit":
        cache = [torch.zeros(shape + (d,), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"]
        cache += [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in "kv"]
    else:
        cache = [torch.zeros(shape + (d,), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    state["spare"] = cache
    state["cache"] = tuple(t[:blocks] for t in cache)
    order = rng.permutation(blocks)[:-(-n // bs)]  # whole blocks in random order, as an allocator hands them out
    slots = (order[:, None] * bs + np.arange(bs)[None, :]).reshape(-1)[:n].astype(np.int64)
    slots[rng.permutation(n)[:_skipped(case)]] = -1
    state["slots"] = torch.as_tensor(slots, device="cuda")
    # stretches of consecutive positions, each from a start of its own
    at, pos = 0, np.empty(n, dtype=np.int64)
    stretch = 1 if n <= 512 else 2048
    while at < n:
        m = min(stretch, n - at, top)
        pos[at:at + m] = rng.integers(0, top - m + 1) + np.arange(m)
        at += m
    state["positions"] = torch.as_tensor(pos, device="cuda")
    state["table"] = _table(top, case["rot"])
    state["half"] = case["style"] == "half"
    q, k, v = (_rows_like((n, h, d), g, _channels(d, g, o)) for h, o in ((hq, False), (hkv, True), (hkv, False)))
    if case["strided"]:  # views of a fused projection's output: [token][query heads | key heads | value heads]
        fused = torch.cat([q, k, v], 1)
        q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    state["q"], state["k"], state["v"] = q, k, v
    state["q_out"] = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
    return state


def _prepare_attention(case, state, g, rng, hq, hkv, d, bs):
    lens, rows = _lengths(case), _rows(case)
    counts = -(-lens // bs)
    if case["op"] == "window":  # blocks that no row sees any more have been given back: their entries are -1
        gone = np.maximum(0, lens - rows - case["window"] + 1) // bs
        kept = -(-case["sinks"] // bs)
    else:
        gone, kept = np.zeros_like(lens), 0
    held = counts - np.maximum(0, gone - kept)
    blocks = int(held.sum()) + 3
    perm = rng.permutation(blocks)
    tables = np.full((len(lens), int(counts.max())), -1, dtype=np.int32)
    at = 0
    for i, c in enumerate(counts):
        e = np.arange(c)
        e = e[(e < kept) | (e >= gone[i])]
        tables[i, e] = perm[at:at + len(e)]
        at += len(e)
    state["cache"] = tuple(torch.empty((blocks, hkv, bs, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    step = max(1, (1 << 26) // (hkv * bs * d))
    for t, outliers in zip(state["cache"], (True, False)):
        ch = _channels(d, g, outliers)
        for b in range(0, blocks, step):
            t[b:b + step] = _rows_like(t[b:b + step].shape, g, ch)
    total = int(rows.sum())
    state["q"] = _rows_like((total, hq, d), g, _channels(d, g, False))
    state["out"] = torch.zeros_like(state["q"])
    state["tables"] = torch.as_tensor(tables, device="cuda")
    state["lens"] = torch.as_tensor(lens.astype(np.int32), device="cuda")
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    state["start_host"], state["lens_host"] = start.tolist(), lens.tolist()  # a scheduler knows both
    state["start"] = torch.as_tensor(start, device="cuda")
    state["max_len"] = int(lens.max())
    state["scale"] = float(np.float32(d ** -0.5))
    state["workspace"] = None
    if case["op"] == "tree":
        state["nodes"] = case["nodes"]
        state["mask"] = torch.as_tensor(_tree_masks(rows, rng), device="cuda")
    else:
        state["window"], state["sinks"], state["single"] = case["window"], case["sinks"], case["chunk"] == 1
    return state


# -------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "rope":
        return _plain_rope(state)
    if state["op"] == "tree":
        return _plain_tree(state)
    return _plain_window_step(state) if state["single"] else _plain_window_chunks(state)


def _run_own(s):
    from paged_kv_cache_276_gb300 import native
    if s["op"] == "rope":
        f = native.pkv_write_rope if len(s["cache"]) == 2 else native.pkv_write_rope_quant
        f(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], s["q_out"], *s["cache"],
          interleaved=not s["half"], d_status=s["status"])
        return (s["q_out"],) + s["cache"]
    hq, d = s["q"].shape[1:]
    n, total, hkv = len(s["lens_host"]), s["q"].shape[0], s["cache"][0].shape[1]
    if s["op"] == "tree":
        if s["workspace"] is None:  # once, as a program keeps it
            size = native.paged_attention_tree_workspace_size(n, total, s["nodes"], hq, hkv, d, s["max_len"])
            s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
        native.paged_attention_tree(s["q"], *s["cache"], s["tables"], s["lens"], s["start"], s["mask"], s["nodes"],
                                    s["max_len"], s["scale"], s["out"], s["workspace"], s["status"])
        return s["out"]
    if s["workspace"] is None:
        size = native.paged_attention_window_workspace_size(n, total, hq, hkv, d, s["max_len"], s["window"],
                                                            s["sinks"])
        s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    native.paged_attention_window(s["q"], *s["cache"], s["tables"], s["lens"], s["max_len"], s["window"], s["sinks"],
                                  s["scale"], s["out"], None if s["single"] else s["start"], s["workspace"],
                                  s["status"])
    return s["out"]


def _rotate(x, c, s, half):
    """x [T, H, d] (fp32), c and s [T, 1, rot / 2]: the first rot values of each row rotated."""
    r = 2 * c.shape[-1]
    y = x.clone()
    if half:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    return y


def _plain_rope(s):
    hkv, bs = s["cache"][0].shape[1:3]
    blocks = s["cache"][0].shape[0]
    c, sn = s["table"][s["positions"]][:, None].chunk(2, -1)
    s["q_out"].copy_(_rotate(s["q"].float(), c, sn, s["half"]))
    slots = torch.where(s["slots"] >= 0, s["slots"], blocks * bs)  # skipped rows land in the block past the pool
    at, off = slots // bs, slots % bs
    rows = (_rotate(s["k"].float(), c, sn, s["half"]), s["v"].float())
    if len(s["cache"]) == 2:
        for x, cache in zip(rows, s["spare"]):
            cache[at, :, off] = x.to(torch.bfloat16)
    else:
        for x, codes, exps in zip(rows, s["spare"][:2], s["spare"][2:]):
            v, e = _quantise(x)
            codes.view(torch.uint8)[at, :, off] = v.view(torch.uint8)
            exps[at, :, off] = e
    return (s["q_out"],) + s["cache"]


def _attend(q, k, v, seen, scale):
    """q [..., R, d], k and v [..., N, d] in fp32, seen [..., R, N]: softmax over the seen keys; none: zeros."""
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, float("-inf"))
    top = z.amax(-1, keepdim=True)
    w = z.sub_(torch.where(top > float("-inf"), top, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, v) / torch.where(total > 0, total, 1.0)


def _plain_tree(s):
    kc, vc = s["cache"]
    hkv, bs, d = kc.shape[1:]
    hq = s["q"].shape[1]
    b, top = s["tables"].shape[0], s["nodes"]
    start, lens = s["start"].long(), s["lens"].long()
    rows = start[1:] - start[:-1]
    node = torch.arange(top, device="cuda")
    real = node[None] < rows[:, None]  # [B, nodes]
    at = torch.where(real, start[:-1, None] + node[None], 0)
    ids = s["tables"].clamp(min=0).long()

    def gather(c):  # [B, blocks, Hkv, bs, d] -> [B, Hkv, tokens, d]
        return c[ids].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)

    q = s["q"].float()[at].reshape(b, top, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    t = torch.arange(ids.shape[1] * bs, device="cuda")
    j = t[None] - (lens - rows)[:, None]  # [B, tokens]: the node that a token is, negative in the context
    bit = (s["mask"][at][:, :, None] >> j.clamp(0, 63)[:, None]) & 1
    inside = (t[None] < lens[:, None])
    seen = (((j < 0)[:, None] | (bit == 1)) & inside[:, None])[:, None, :, None]  # [B, 1, nodes, 1, tokens]
    seen = seen.expand(b, 1, top, hq // hkv, t.numel()).reshape(b, 1, -1, t.numel())
    v = gather(vc).masked_fill_(~inside[:, None, :, None], 0.0)
    o = _attend(q, gather(kc), v, seen, s["scale"])
    o = o.reshape(b, hkv, top, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, top, hq, d)
    s["out"].copy_(o[real])
    return s["out"]


def _plain_window_step(s):
    kc, vc = s["cache"]
    hkv, bs, d = kc.shape[1:]
    b, hq = s["q"].shape[:2]
    lens = s["lens"].long()[:, None]
    first = torch.arange(s["sinks"], device="cuda")[None].expand(b, -1)
    recent = lens - 1 - torch.arange(min(s["window"], s["max_len"]), device="cuda")[None]
    pos = torch.cat([first, recent], 1)  # the sinks, then the window
    sink = torch.cat([torch.ones_like(first), torch.zeros_like(recent)], 1).bool()
    seen = torch.where(sink, (pos < lens) & (pos <= lens - 1 - s["window"]), pos >= 0)  # a sink in the window once
    pos = torch.where(seen, pos, 0)
    ids = torch.gather(s["tables"].long(), 1, pos // bs)
    seen_rows = seen[:, None, :, None]
    ids = torch.where(seen, ids, 0)

    def gather(c):  # [B, N, Hkv, d] -> [B, Hkv, N, d]
        return c[ids, :, pos % bs].float().transpose(1, 2)

    q = s["q"].float().reshape(b, hkv, hq // hkv, d)
    v = gather(vc).masked_fill_(~seen_rows, 0.0)
    s["out"].copy_(_attend(q, gather(kc), v, seen[:, None, None], s["scale"]).reshape(b, hq, d))
    return s["out"]


def _plain_window_chunks(s):
    kc, vc = s["cache"]
    hkv, bs, d = kc.shape[1:]
    hq = s["q"].shape[1]
    w, sinks = s["window"], s["sinks"]
    for i, n in enumerate(s["lens_host"]):
        a, e = s["start_host"][i], s["start_host"][i + 1]
        ctx = n - (e - a)
        for r in range(a, e, 1024):  # a stretch of queries with the keys that any of them sees
            r1 = min(e, r + 1024)
            p = torch.arange(ctx + r - a, ctx + r1 - a, device="cuda")
            lo = max(0, ctx + r - a - w + 1)
            t = torch.cat([torch.arange(min(sinks, lo), device="cuda"), torch.arange(lo, ctx + r1 - a, device="cuda")])
            at, off = s["tables"][i].long()[t // bs], t % bs
            seen = (t[None] <= p[:, None]) & ((t[None] > p[:, None] - w) | (t[None] < sinks))
            k, v = (c[at, :, off].float().transpose(0, 1) for c in (kc, vc))  # [Hkv, N, d]
            q = s["q"][r:r1].float().reshape(r1 - r, hkv, hq // hkv, d).permute(1, 2, 0, 3)  # [Hkv, G, R, d]
            o = _attend(q, k[:, None], v[:, None], seen, s["scale"])
            s["out"][r:r1] = o.permute(2, 0, 1, 3).reshape(r1 - r, hq, d).to(torch.bfloat16)
    return s["out"]


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definition in 64 bits, token by token of the append, sequence by sequence of the attention."""
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_attention(case, s)


def _exact_rope(case, s):
    d, r, bs = case["head_dim"], case["rot"], case["block"]
    angles = s["table"].to(torch.float64)[s["positions"]]
    z = torch.complex(angles[:, :r // 2], angles[:, r // 2:])[:, None]  # cos + i sin

    def turned(x):
        y = x.to(torch.float64)
        if case["style"] == "half":
            w = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * z
            return torch.cat([w.real, w.imag, y[..., r:]], -1)
        w = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * z
        return torch.cat([torch.view_as_real(w).flatten(-2), y[..., r:]], -1)

    live = (s["slots"] >= 0).nonzero()[:, 0]
    at, off = s["slots"][live] // bs, s["slots"][live] % bs
    got = []
    for x, cache in zip((turned(s["k"])[live], s["v"][live].to(torch.float64)), s["cache"]):
        y = cache.to(torch.float64)
        if case["cache"] == "8bit":  # what the codes round: the row over its power of two
            a = x.abs().amax(-1, keepdim=True)
            x = x * torch.exp2(-torch.ceil(torch.log2(a.clamp(min=2.0 ** -300) / 448.0) - 1e-12).clamp(-31, 31))
        y[at, :, off] = x
        got.append(y)
    return (turned(s["q"]),) + tuple(got) + ((None, None) if case["cache"] == "8bit" else ())


def _exact_attention(case, s):
    hkv, bs = case["kv_heads"], case["block"]
    hq, d = s["q"].shape[1:]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if work(case)["flops"] > 5e12:
        return None  # at the card's rate in 64 bits more than some seconds
    for i, n in enumerate(s["lens_host"]):
        a, e = s["start_host"][i], s["start_host"][i + 1]
        for r in range(a, e, 256):
            r1 = min(e, r + 256)
            p = torch.arange(n - (e - r), n - (e - r1), device="cuda")  # the rows' positions
            if case["op"] == "tree":
                t = torch.arange(n, device="cuda")
                j = t - (n - (e - a))
                words = s["mask"][r:r1, None]
                seen = (j < 0)[None] | (((words >> j.clamp(min=0)[None]) & 1) == 1)
            else:
                far = p[:, None] - torch.arange(n, device="cuda")[None]  # how far back a key lies
                seen = (far >= 0) & ((far < case["window"]) | (torch.arange(n, device="cuda")[None] < case["sinks"]))
                t = seen.any(0).nonzero()[:, 0]
                seen = seen[:, t]
            rows = s["tables"][i].long()[t // bs]
            k, v = (c[rows, :, t % bs].to(torch.float64) for c in s["cache"])  # [N, Hkv, d]
            q = s["q"][r:r1].to(torch.float64).reshape(r1 - r, hkv, hq // hkv, d)
            z = torch.einsum("rhgd,thd->hgrt", q, k) * s["scale"]
            z = z.masked_fill(~seen, float("-inf"))
            o = torch.einsum("hgrt,thd->rhgd", torch.softmax(z, -1), v)
            out[r:r1] = o.reshape(r1 - r, hq, d)
    return out
