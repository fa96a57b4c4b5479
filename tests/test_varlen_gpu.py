"""attn_fwd_varlen: packed sequences of different lengths, against 64-bit attention of each
sequence by itself."""
import math

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import DT, causal, close, offsets, plain

pytestmark = pytest.mark.gpu


def make(total, Hq, Hkv, D, dtype, layout="packed", std=1.0, seed=0, total_k=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    total_k = total if total_k is None else total_k

    def rows(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])

    if layout == "fused":  # cut from one projection's output
        x = rows(total, Hq + 2 * Hkv, D)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if layout == "heads":  # [heads, rows, D] seen as [rows, heads, D]
        return (rows(Hq, total, D).transpose(0, 1), rows(Hkv, total_k, D).transpose(0, 1),
                rows(Hkv, total_k, D).transpose(0, 1))
    return rows(total, Hq, D), rows(total_k, Hkv, D), rows(total_k, Hkv, D)


def check(q, k, v, o, lse, lens, lens_k, dtype, scale, is_causal):
    Hq, G = q.shape[1], q.shape[1] // k.shape[1]
    a = b = 0
    for s, (nq, nk) in enumerate(zip(lens, lens_k)):
        see = causal(nq, nk) if is_causal else torch.ones(nq, nk, dtype=torch.bool)
        for h in range(Hq):
            ro, rl, to, tl = plain(q[a:a + nq, h], k[b:b + nk, h // G], v[b:b + nk, h // G], see, scale, dtype)
            close(o[a:a + nq, h], ro, to, f"O of sequence {s}, head {h}")
            if lse is not None:
                close(lse[h, a:a + nq], rl, tl, f"LSE of sequence {s}, head {h}")
        a, b = a + nq, b + nk


CASES = [
    # lens, Hq, Hkv, D, dtype, causal, layout, std of q, k, v
    ([1], 1, 1, 64, "f16", True, "packed", 1.0),
    ([1], 4, 1, 128, "bf16", False, "packed", 1.0),
    ([37], 2, 1, 64, "f16", True, "packed", 1.0),
    ([128], 2, 2, 128, "bf16", True, "packed", 1.0),
    ([129, 1, 0, 255, 256, 257], 4, 2, 128, "bf16", True, "packed", 1.0),
    ([129, 1, 0, 255, 256, 257], 4, 2, 64, "f16", True, "fused", 1.0),
    ([129, 1, 0, 255, 256, 257], 3, 1, 128, "f16", True, "heads", 1.0),
    ([129, 1, 0, 255, 256, 257], 3, 3, 64, "bf16", False, "packed", 1.0),
    ([0, 0, 5], 2, 1, 128, "f16", True, "packed", 1.0),
    ([0, 300, 0, 40, 513, 0], 8, 1, 128, "bf16", True, "fused", 1.0),
    ([300, 40, 513, 127, 640], 6, 2, 64, "bf16", False, "heads", 1.0),
    ([300, 40, 513], 8, 2, 128, "bf16", True, "packed", 4.0),
    ([700, 2], 5, 5, 128, "f16", True, "packed", 2.0),
    ([1 + (7 * i) % 11 for i in range(200)], 2, 1, 64, "bf16", True, "packed", 1.0),
    ([(5 * i) % 3 for i in range(2500)], 2, 1, 64, "f16", True, "packed", 1.0),
    ([(5 * i) % 3 for i in range(2500)], 1, 1, 64, "f16", False, "packed", 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-" + "-".join(map(str, c[1:])))
def test_packed_sequences(case):
    lens, Hq, Hkv, D, dtype, is_causal, layout, std = case
    q, k, v = make(sum(lens), Hq, Hkv, D, dtype, layout, std, seed=len(lens) + Hq + D)
    o, lse = binding.attention_varlen(q, k, v, offsets(lens), causal=is_causal)
    assert binding.attn_last_device_error(torch.cuda.current_stream()) == binding.ATTN_OK
    check(q, k, v, o, lse, lens, lens, dtype, 1 / math.sqrt(D), is_causal)


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("is_causal", [True, False])
def test_queries_and_keys_of_different_lengths(Hq, Hkv, is_causal):
    """Chunks over longer keys, offsets that are no multiple of a tile, more queries than keys
    (rows that see nothing), no keys, no queries."""
    lens_q = [64, 1, 130, 200, 300, 5, 0, 140, 257]
    lens_k = [320, 513, 131, 200, 100, 0, 40, 1, 400]
    q, k, v = make(sum(lens_q), Hq, Hkv, 128, "bf16", seed=3, total_k=sum(lens_k))
    o, lse = binding.attention_varlen(q, k, v, offsets(lens_q), offsets(lens_k), causal=is_causal, scale=0.11)
    assert binding.attn_last_device_error(torch.cuda.current_stream()) == binding.ATTN_OK
    check(q, k, v, o, lse, lens_q, lens_k, "bf16", 0.11, is_causal)


def test_no_keys_at_all():
    q = make(20, 4, 2, 64, "f16")[0]
    none = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    o, lse = binding.attention_varlen(q, none, none, offsets([12, 8]), offsets([0, 0]))
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


def test_rows_behind_the_last_sequence_and_other_sequences_stay_out():
    """Padding rows hold NaN, one sequence is NaN all over: neither reaches another, and the
    outputs' padding rows are left as they were."""
    lens, pad = [200, 77, 130, 1, 300], 100
    total = sum(lens)
    for Hq, Hkv in ((4, 2), (3, 1)):
        q, k, v = make(total + pad, Hq, Hkv, 128, "bf16", seed=5)
        for x in (q, k, v):
            x[total:] = math.nan
            x[277:407] = math.nan  # the third sequence
        v[total + 1:] = math.inf
        for is_causal in (True, False):
            o = torch.full_like(q, 7.0)
            lse = torch.full((Hq, total + pad), 8.0, device="cuda")
            binding.attention_varlen(q, k, v, offsets(lens), causal=is_causal, out=o, lse_out=lse)
            assert bool((o[total:] == 7).all()) and bool((lse[:, total:] == 8).all())
            assert bool(torch.isnan(o[277:407]).all())
            at = [0, 200, 277, 407, 408]
            for i, (a, n) in enumerate(zip(at, lens)):
                if i != 2:
                    check(q[a:a + n], k[a:a + n], v[a:a + n], o[a:a + n], lse[:, a:a + n], [n], [n], "bf16",
                          1 / math.sqrt(128), is_causal)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 128, "bf16"), (3, 3, 64, "f16")])
def test_non_finite_values_reach_the_rows_that_see_them(Hq, Hkv, D, dtype):
    """Infinities and NaN in V, and NaN in K, behind the causal mask: rows before them are as
    without them, rows from them on get what the sum over their keys gives."""
    lens = [190, 260]
    q, k, v = make(sum(lens), Hq, Hkv, D, dtype, seed=9)
    v[150, :, 3] = math.inf
    v[170, 0, 5] = math.nan
    v[188, :, D - 1] = -math.inf
    v[190 + 255, :, 0] = math.nan
    o, lse = binding.attention_varlen(q, k, v, offsets(lens))
    check(q, k, v, o, lse, lens, lens, dtype, 1 / math.sqrt(D), True)
    q, k, v = make(sum(lens), Hq, Hkv, D, dtype, seed=10)
    k[190 + 200:] = math.nan
    o, lse = binding.attention_varlen(q, k, v, offsets(lens))
    for h in range(Hq):  # the second sequence's first 200 rows see finite keys only
        ro, rl, to, tl = plain(q[190:390, h], k[190:390, h // (Hq // Hkv)], v[190:390, h // (Hq // Hkv)],
                               causal(200, 200), 1 / math.sqrt(D), dtype)
        close(o[190:390, h], ro, to, "O before the NaN keys")
        close(lse[h, 190:390], rl, tl, "LSE before the NaN keys")
    assert bool(torch.isnan(o[390:]).all())


def test_equal_lengths_agree_with_the_batched_call():
    """Four sequences of one length: the same rows as attn_fwd within both calls' bounds, on a
    length past a few tiles (every element, long rows)."""
    B, N, Hq, Hkv, D = 4, 1500, 8, 2, 128
    q, k, v = make(B * N, Hq, Hkv, D, "bf16", seed=21)
    o, lse = binding.attention_varlen(q, k, v, offsets([N] * B))

    def heads(x):
        return x.view(B, N, x.shape[1], D).transpose(1, 2).contiguous()

    o2, lse2 = binding.attention(heads(q), heads(k), heads(v))
    o2 = o2.transpose(1, 2).reshape(B * N, Hq, D)
    lse2 = lse2.transpose(0, 1).reshape(Hq, B * N)
    u = 2.0 ** -8
    # each is off by at most u (|O| + A) + small, with A <= max |v| of the sequence
    amax = float(v.abs().max())
    assert float((o.float() - o2.float()).abs().max()) <= 2 * (2 * u + 2.0 ** -12) * amax
    assert float((lse - lse2).abs().max()) <= 2.0 ** -12


def test_long_sequence_every_block_of_one_head():
    """A 9000-token prompt beside a short one: rows around every 128-row border."""
    lens = [9000, 50]
    q, k, v = make(sum(lens), 4, 1, 128, "bf16", seed=22)
    o, lse = binding.attention_varlen(q, k, v, offsets(lens))
    rows = sorted({min(8999, 128 * i + d) for i in range(71) for d in (0, 127)})
    see = causal(9000, 9000)[rows]
    for h in (0, 3):
        ro, rl, to, tl = plain(q[rows, h], k[:9000, 0], v[:9000, 0], see, 1 / math.sqrt(128), "bf16")
        close(o[rows, h], ro, to, "O")
        close(lse[h, rows], rl, tl, "LSE")


def test_same_bits_twice_without_lse_and_on_another_stream():
    lens = [300, 20, 600]
    q, k, v = make(sum(lens), 8, 2, 128, "f16", "fused", seed=23)
    cu = offsets(lens)
    o1, _ = binding.attention_varlen(q, k, v, cu)
    o2, none = binding.attention_varlen(q, k, v, cu, with_lse=False)
    assert none is None and torch.equal(o1, o2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o3, lse3 = binding.attention_varlen(q, k, v, cu, stream=s)
    s.synchronize()
    assert torch.equal(o1, o3)
    # an output with strides of its own
    wide = torch.zeros((sum(lens), 12, 128), dtype=torch.float16, device="cuda")
    binding.attention_varlen(q, k, v, cu, out=wide[:, 2:10])
    assert torch.equal(wide[:, 2:10], o1) and bool((wide[:, :2] == 0).all()) and bool((wide[:, 10:] == 0).all())


def test_captured_call_replays_on_new_lengths():
    q, k, v = make(700, 4, 2, 64, "bf16", seed=24)
    cu = offsets([700, 0, 0])
    o, lse = torch.zeros_like(q), torch.zeros((4, 700), device="cuda")
    binding.attention_varlen(q, k, v, cu, out=o, lse_out=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.attention_varlen(q, k, v, cu, out=o, lse_out=lse)
    for lens in ([100, 500, 100], [1, 0, 699], [256, 256, 188]):
        cu.copy_(offsets(lens))
        q.copy_(make(700, 4, 2, 64, "bf16", seed=sum(lens[:1]))[0])
        g.replay()
        torch.cuda.synchronize()
        check(q, k, v, o, lse, lens, lens, "bf16", 1 / 8, True)


def test_bad_offsets_are_clamped_and_reported():
    """Offsets past the tensors or descending: no access outside them, the error word says so,
    and the next call is right."""
    q, k, v = make(300, 4, 2, 128, "bf16", seed=25)
    s = torch.cuda.current_stream()
    for cu in ([0, 100, 5000], [0, 200, 100, 300], [-7, 50, 300]):
        binding.attention_varlen(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert binding.attn_last_device_error(s) == binding.ATTN_ERR_SHAPE
    o, lse = binding.attention_varlen(q, k, v, offsets([100, 200]))
    assert binding.attn_last_device_error(s) == binding.ATTN_OK
    check(q, k, v, o, lse, [100, 200], [100, 200], "bf16", 1 / math.sqrt(128), True)


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
def test_overlapping_offsets_do_no_more_work_than_ascending_ones(Hq, Hkv):
    """Offsets that go back and forth over the rows ask for more blocks than the tensors hold:
    clamped, cut and reported, and the next call is right."""
    q, k, v = make(300, Hq, Hkv, 64, "f16", seed=27)
    s = torch.cuda.current_stream()
    cu = torch.tensor([0, 300] * 40, dtype=torch.int32, device="cuda")
    binding.attention_varlen(q, k, v, cu)
    assert binding.attn_last_device_error(s) == binding.ATTN_ERR_SHAPE
    o, lse = binding.attention_varlen(q, k, v, offsets([100, 200]))
    assert binding.attn_last_device_error(s) == binding.ATTN_OK
    check(q, k, v, o, lse, [100, 200], [100, 200], "f16", 1 / 8, True)


def test_timeout_is_reported_and_the_next_call_works():
    lib = binding.load()
    q, k, v = make(300, 4, 2, 128, "bf16", seed=26)
    s = torch.cuda.current_stream()
    binding.attention_varlen(q, k, v, offsets([300]))
    torch.cuda.synchronize()
    try:
        lib.attn_test_set_wait_timeout_ns(50_000_000)
        lib.attn_test_inject_stall(1)
        binding.attention_varlen(q, k, v, offsets([300]))
        assert binding.attn_last_device_error(s) == binding.ATTN_ERR_TIMEOUT
    finally:
        lib.attn_test_inject_stall(0)
        lib.attn_test_set_wait_timeout_ns(0)
    o, lse = binding.attention_varlen(q, k, v, offsets([300]))
    assert binding.attn_last_device_error(s) == binding.ATTN_OK
    check(q, k, v, o, lse, [300], [300], "bf16", 1 / math.sqrt(128), True)
