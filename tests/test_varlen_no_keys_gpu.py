"""attn_fwd_varlen where many units have no keys: rows that see none get O = 0 and LSE = -inf, the
others what they get without them."""
import math

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import DT, causal, close, offsets, plain

pytestmark = pytest.mark.gpu

CASES = [
    # query lengths, key lengths, Hq, Hkv, D, dtype, causal
    ([8192], [512], 32, 8, 128, "bf16", True),
    ([6144], [1024], 32, 8, 128, "bf16", True),
    ([100] * 41, [300] + [0] * 40, 32, 8, 128, "bf16", False),
    ([1] * 64, [0] * 40 + [700] * 8 + [0] * 16, 32, 8, 128, "bf16", True),
    ([6000, 130], [200, 0], 6, 2, 64, "f16", True),
    ([700, 260, 5, 130] * 20, [1, 300, 0, 131] * 20, 8, 2, 64, "bf16", True),
    ([40] * 300, [0, 0, 0, 17, 0] * 60, 6, 6, 128, "f16", False),
    ([1 + i % 3 for i in range(2500)], [i % 2 for i in range(2500)], 8, 8, 64, "f16", True),
    ([300] * 30, [0] * 29 + [1], 32, 8, 128, "f16", True),
]


def rows(n, heads, D, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((n, heads, D), generator=g, device="cuda").to(DT[dtype])


def check(q, k, v, o, lse, lens_q, lens_k, dtype, is_causal):
    G = q.shape[1] // k.shape[1]
    a = b = 0
    for s, (nq, nk) in enumerate(zip(lens_q, lens_k)):
        blind = min(nq, max(0, nq - nk)) if is_causal or nk == 0 else 0  # rows that see no key
        assert bool((o[a:a + blind] == 0).all()) and bool((lse[:, a:a + blind] == -math.inf).all()), f"sequence {s}"
        if blind < nq:
            see = causal(nq, nk)[blind:] if is_causal else torch.ones(nq, nk, dtype=torch.bool)
            for h in (0, q.shape[1] - 1):
                ro, rl, to, tl = plain(q[a + blind:a + nq, h], k[b:b + nk, h // G], v[b:b + nk, h // G], see,
                                       1 / math.sqrt(q.shape[2]), dtype)
                close(o[a + blind:a + nq, h], ro, to, f"O of sequence {s}, head {h}")
                close(lse[h, a + blind:a + nq], rl, tl, f"LSE of sequence {s}, head {h}")
        a, b = a + nq, b + nk


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{sum(c[0])}over{sum(c[1])}-" + "-".join(map(str, c[2:])))
def test_units_without_keys(case):
    lens_q, lens_k, Hq, Hkv, D, dtype, is_causal = case
    q = rows(sum(lens_q) + 2, Hq, D, dtype, 61)
    k, v = (rows(sum(lens_k) + 1, Hkv, D, dtype, 62 + i) for i in range(2))
    o = torch.full_like(q, 7.0)
    lse = torch.full((Hq, q.shape[0]), 8.0, device="cuda")
    binding.attention_varlen(q, k, v, offsets(lens_q), offsets(lens_k), causal=is_causal, out=o, lse_out=lse)
    assert binding.attn_last_device_error(torch.cuda.current_stream()) == binding.ATTN_OK
    check(q, k, v, o, lse, lens_q, lens_k, dtype, is_causal)
    assert bool((o[-2:] == 7).all()) and bool((lse[:, -2:] == 8).all())


def test_captured_call_replays_with_and_without_keys():
    """One graph over 1200 queries: keys for all of them, for the last rows, for one sequence of
    three, for none, and for all again."""
    q, k, v = rows(1200, 32, 128, "bf16", 71), rows(1200, 8, 128, "bf16", 72), rows(1200, 8, 128, "bf16", 73)
    cu_q, cu_k = offsets([1200, 0, 0]), offsets([1200, 0, 0])
    o, lse = torch.zeros_like(q), torch.zeros((32, 1200), device="cuda")
    binding.attention_varlen(q, k, v, cu_q, cu_k, out=o, lse_out=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.attention_varlen(q, k, v, cu_q, cu_k, out=o, lse_out=lse)
    for lens_q, lens_k in (([1200, 0, 0], [60, 0, 0]), ([500, 400, 300], [0, 333, 0]), ([400] * 3, [0] * 3),
                           ([500, 400, 300], [500, 400, 300])):
        cu_q.copy_(offsets(lens_q))
        cu_k.copy_(offsets(lens_k))
        g.replay()
        torch.cuda.synchronize()
        check(q, k, v, o, lse, lens_q, lens_k, "bf16", True)
    assert binding.attn_last_device_error(torch.cuda.current_stream()) == binding.ATTN_OK
