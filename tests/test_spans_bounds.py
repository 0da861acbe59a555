"""The bound of the windowed and tree attention's GPU tests on marked values, without a GPU: it passes the oracle's
own answer rounded to bf16 and fails an answer that lacks one key tile or counts one twice."""
import numpy as np
import pytest
import torch

from oracle import quant as OQ
from oracle import spans as OS
from test_gpu_spans import check


def bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("d,L,tile", [(64, 40000, 32), (64, 30000, 64), (128, 30000, 64), (128, 40000, 32)])
def test_a_lost_tile_passes_the_bound(d, L, tile, flat):
    rng = np.random.default_rng(1)
    q, k = (bf16(rng.standard_normal(s)).view(torch.int16).numpy().view(np.uint16) for s in ((1, 2, d), (1, 1, L, d)))
    if flat:
        q = np.zeros_like(q)
    v = np.zeros((1, 1, L, d), np.uint16)
    v[0, 0, np.arange(L), np.arange(L) // tile % d] = 0x3F80
    args = (q, k, v, np.zeros((1, 1), np.int32), [L], [0, 1], float(np.float32(d ** -0.5)))
    every = np.ones((1, L), bool)
    ref, mag, dot = OS.attend(*args, [every])

    def verdict(out):
        check(bf16(out).view(torch.int16).numpy().view(np.uint16), ref, mag, dot, L, d)

    verdict(ref)
    # its numerator and denominator with tile x taken `times` times
    s = OQ.bf16_values(q)[0] @ OQ.bf16_values(k)[0, 0].T * args[-1]
    w, values = np.exp(s - s.max(-1, keepdims=True)), OQ.bf16_values(v)[0, 0]
    for x in rng.choice(L // tile, 12, replace=False):
        part = slice(x * tile, (x + 1) * tile)
        for times in (0, 2):
            more = (times - 1) * w[:, part]
            out = (w @ values + more @ values[part]) / (w.sum(-1) + more.sum(-1))[:, None]
            with pytest.raises(AssertionError, match="times the bound"):
                verdict(out[None])
