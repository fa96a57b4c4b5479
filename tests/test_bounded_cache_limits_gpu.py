"""The window, weighing and eviction calls at the ends of what they take: the widest table, offsets
past 32 bits, more large units than are dealt one by one, and what a wait that ran out leaves.

Bound of a sum of weights, from the order in which kv_weigh_kernel adds (f = 2^-24): the terms are off
as test_weigh_evict_gpu says.  A warpgroup has 64 columns of a row tile, in 4 chains of 16 that 2 sums
join, and one sum per row tile; the two warpgroups' sums are added once, and the old value once more:
(16 + 2 + tiles + 2) f of the sum."""
import math

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import F, close, offsets
from paged_util import build, gather
from test_tree_gpu import i32, queries, status, trees
from test_weigh_evict_gpu import logsumexps
from test_window_gpu import check_trees

pytestmark = pytest.mark.gpu


def weights_in_64_bits(q, lse, k, scale):
    """Sums [Hkv, n] that q [T, Hq, D], lse [Hq, T] give the keys k [n, Hkv, D], and their bounds."""
    n, Hkv, D = k.shape
    T, G = q.shape[0], q.shape[1] // Hkv
    q = q.double().view(T, Hkv, G, D).permute(1, 2, 0, 3)
    k, l = k.double().permute(1, 2, 0)[:, None], lse.double().view(Hkv, G, T, 1)
    s = q @ k * scale
    e = (D + 2) * F * (q.abs() @ k.abs()) * scale
    see = torch.ones(T, n, dtype=torch.bool, device=q.device).tril(n - T)
    p = torch.where(see, torch.exp(s - l), 0.0)
    d = e + F * s.abs() + 2 * F * l.abs() + F * (s - l).abs() + 2.0 ** -22
    tiles = -(-T // (128 // G))
    sums = p.sum((1, 2))
    return sums.cpu(), ((p * d * (1 + d)).sum((1, 2)) + (20 + tiles) * F * sums + 1e-30).cpu()


def test_more_large_units_than_are_dealt_one_by_one():
    """A group of 65 heads leaves one token to a row tile: ten times as many units of 8 row tiles and more
    as there are SMs, of which the first eighty percent are dealt one by one, and units of fewer behind them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hkv, G, D, scale = 2, 65, 64, 0.125
    blocks = -(-10 * sms // (24 * Hkv))
    lens = [256 * blocks + 16 + 3 * i for i in range(24)] + [700 + i for i in range(8)]
    T = [8 + i % 5 for i in range(24)] + [1 + i % 7 for i in range(8)]
    cache = build(lens, 64, Hkv, D, "bf16", seed=91)
    q = queries(sum(T), Hkv * G, D, "bf16", 92)
    lse, a = torch.empty((Hkv * G, sum(T)), device="cuda"), 0
    for s, t in enumerate(T):
        lse[:, a:a + t] = logsumexps(q[a:a + t], gather(cache, s)[0], t, scale)
        a += t
    weights = torch.full_like(cache.weights(), -3.0)
    binding.kv_weigh(cache, weights, q, lse, offsets(T), accumulate=False)
    assert status() == binding.ATTN_OK
    a = 0
    for s, (n, t) in enumerate(zip(lens, T)):
        want, tol = weights_in_64_bits(q[a:a + t], lse[:, a:a + t], gather(cache, s)[0], scale)
        close(weights[0, s, :, :n], want, tol, f"sequence {s}")
        assert bool((weights[0, s, :, n:] == -3).all())
        a += t


@pytest.mark.parametrize("window,sinks", [(None, 0), (None, 300), (1, None), (700, None), (None, None)])
def test_windows_of_the_widest_table(window, sinks):
    """None: one less than the table's positions, the largest value that is not the plain call's."""
    page, width = 4096, (2 ** 30 - 1) // 4096
    cache = build([5000, 40], page, 2, 64, "f16", seed=93, width=width)
    most, T = page * width - 1, [9, 1]
    window, sinks = (most if x is None else x for x in (window, sinks))
    par = trees(T, 94)
    q = queries(10, 4, 64, "f16", 95)
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=i32([x for p in par for x in p]), window=window, sinks=sinks)
    assert status() == binding.ATTN_OK
    check_trees(q, cache, o, lse, range(2), par, "f16", 1 / 8, window, sinks)


def test_offsets_beyond_32_bits():
    """The last pages of pools of 2.5e9 elements a layer, and the last row of 2^31 weights."""
    layers, n_pages, Hkv, page, D, n_rows, width = 2, 600, 8, 4096, 128, 8, 4096
    n, row, T, scale = 9000, 7, 3, 1 / math.sqrt(128)
    cache = binding.KVPages.empty(layers, n_pages, Hkv, page, D, n_rows, width, torch.bfloat16)
    g = torch.Generator(device="cuda")
    g.manual_seed(96)
    pages = [599, 597, 598]
    for x in (cache.k, cache.v):
        for p in pages:
            x[:, p] = torch.randn((layers, Hkv, page, D), generator=g, device="cuda").to(x.dtype)
    cache.table[row, :3] = i32(pages)
    cache.lens[row] = n
    cache.refs[597:] = 1
    q, seqs = queries(T, Hkv, D, "bf16", 97), i32([row])
    o, lse = binding.attention_tree(q, cache, offsets([T]), seqs=seqs, layer=1, window=1500, sinks=7)
    assert status() == binding.ATTN_OK
    check_trees(q, cache, o, lse, [row], [[-1, 0, 1]], "bf16", scale, 1500, 7, layer=1)
    o, lse = binding.attention_tree(q, cache, offsets([T]), seqs=seqs, layer=1)
    weights = cache.weights()
    assert weights.numel() == 2 ** 31
    weights[1, row, :, :n - T] = 0.5
    binding.kv_weigh(cache, weights, q, lse, offsets([T]), seqs=seqs, layer=1)
    assert status() == binding.ATTN_OK
    want, tol = weights_in_64_bits(q, lse, gather(cache, row, 1)[0], scale)
    want[:, :n - T] += 0.5
    close(weights[1, row, :, :n], want, tol + F * want, "weights")
    weights[0, row, :, :n] = torch.rand((Hkv, n), generator=g, device="cuda")
    w = weights[:, row, :, :n].clone()
    old = [torch.stack([x.transpose(0, 1) for x in pair]) for pair in zip(*(gather(cache, row, i) for i in (0, 1)))]
    sinks, heavy, recent = 5, 4000, 300
    binding.kv_evict(cache, seqs, weights, sinks=sinks, heavy=heavy, recent=recent)
    assert status() == binding.ATTN_OK
    keep = sinks + heavy + recent
    best = torch.sort(w[:, :, sinks:n - recent], dim=-1, descending=True, stable=True).indices[:, :, :heavy] + sinks
    at = torch.arange(n, device="cuda").expand(layers, Hkv, n)
    src = torch.cat([at[:, :, :sinks], best.sort(-1).values, at[:, :, n - recent:]], -1)
    new = [torch.stack([x.transpose(0, 1) for x in pair]) for pair in zip(*(gather(cache, row, i) for i in (0, 1)))]
    for a, b in zip(old, new):
        assert torch.equal(torch.gather(a, 2, src[..., None].expand(-1, -1, -1, D)), b)
    assert torch.equal(weights[:, row, :, :keep], torch.gather(w, 2, src)) and not bool(weights[:, row, :, keep:].any())
    assert not bool(weights[:, :row].any())
    assert cache.lens.tolist() == [0] * 7 + [keep] and cache.table[row, :3].tolist() == [599, 597, -1]
    assert cache.refs[597:].tolist() == [1, 0, 1]


def test_sums_that_a_wait_cut_short_are_restored_and_added_again():
    """A call that gave up leaves undefined the sums of the listed sequences, in its layer, and no others."""
    lens, T = [900, 300, 400], [40, 3]
    cache = build(lens, 64, 2, 128, "bf16", n_layers=2, seed=98)
    q, lse, seqs = queries(43, 8, 128, "bf16", 99), torch.full((8, 43), 6.0, device="cuda"), i32([2, 0])
    weights, lib = cache.weights().uniform_(0.0, 2.0), binding.load()
    before, good = weights.clone(), weights.clone()
    binding.kv_weigh(cache, good, q, lse, offsets(T), seqs=seqs, layer=1)
    assert status() == binding.ATTN_OK
    try:
        lib.attn_test_set_wait_timeout_ns(20_000_000)
        lib.attn_test_inject_stall(1)
        binding.kv_weigh(cache, weights, q, lse, offsets(T), seqs=seqs, layer=1)
    finally:
        lib.attn_test_inject_stall(0)
        lib.attn_test_set_wait_timeout_ns(0)
    assert status() == binding.ATTN_ERR_TIMEOUT
    assert torch.equal(weights[0], before[0]) and torch.equal(weights[1, 1], before[1, 1])
    for s in (0, 2):
        assert torch.equal(weights[1, s, :, lens[s]:], before[1, s, :, lens[s]:])
    weights.copy_(before)
    binding.kv_weigh(cache, weights, q, lse, offsets(T), seqs=seqs, layer=1)
    assert status() == binding.ATTN_OK and torch.equal(weights, good)


def test_a_sequence_that_fills_the_widest_table():
    """2^30 positions over one page that every entry names: each of its rows stands for as many equal keys as
    a token sees of them.  Attention with windows, weights of every position, and a cut to 5093 of them,
    which moves the rows of the shared page into the sequence's own first two."""
    page, width, D, scale, T = 4096, (2 ** 30 - 1) // 4096, 64, 1 / 8, 2
    n = page * width - 3  # a last page that is not full
    i = dict(dtype=torch.int32, device="cuda")
    cache = binding.KVPages.empty(1, 3, 1, page, D, 1, width, torch.float16)
    g = torch.Generator(device="cuda")
    g.manual_seed(101)
    for x in (cache.k, cache.v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    cache.table.zero_()
    cache.lens.fill_(n)
    cache.refs.copy_(torch.tensor([width, 0, 0], **i))
    q = queries(T, 2, D, "f16", 102)
    rows = torch.arange(page, device="cuda")

    def copies(a, b):
        """How often each row of the page stands in positions [a, b)."""
        return ((b - rows + page - 1) // page - (a - rows + page - 1) // page).double()

    s = torch.einsum("thd,rd->thr", q.double(), cache.k[0, 0, 0].double()) * scale
    most = float(s.abs().max())
    e = (D + 2) * F * float((q.double().abs() @ cache.k[0, 0, 0].double().abs().T).max()) * scale
    lse = None
    for window, sinks in ((1, 0), (5000, 777), (n // 2 + 9, 10 ** 6 + 1), (n - 5, 3), (None, 0)):
        o, lse = binding.attention_tree(q, cache, offsets([T]), window=window, sinks=sinks)
        assert status() == binding.ATTN_OK
        for t in range(T):
            pos = n - T + t
            lo = 0 if window is None else max(0, pos - window + 1)
            seen = copies(lo, pos + 1) + copies(0, min(sinks, lo))
            want = torch.logsumexp(s[t] + seen.log(), -1)
            p = torch.exp(s[t] - want[:, None]) * seen
            ref, size = p @ cache.v[0, 0, 0].double(), p @ cache.v[0, 0, 0].double().abs()
            # the bounds of packed_util over so many keys and 152 pieces; an fp16 weight below the smallest
            # normal number is off by 2^-25 of the row's largest, so each copy of a row by that in all
            count, u = float(seen.sum()), 2.0 ** -11
            add = (72 + count / 128 + 152 + 8) * F + 2.0 ** -21
            tiny = 2.0 ** -25 * count / torch.exp(want - s[t].amax(-1))[:, None] * float(cache.v[0, 0].abs().max())
            close(o[t], ref.cpu(), (u * ref.abs() + (1 + u) * (u + 2 * (e + 4 * F * most) + 2 * add) * size + tiny + 2.0 ** -25).cpu(),
                  f"O of token {t}, window {window}")
            close(lse[:, t], want.cpu(), (e + (8 * most + 2 * want.abs()) * F + add).cpu(), f"LSE of token {t}, window {window}")
    weights = cache.weights()
    binding.kv_weigh(cache, weights, q, lse, offsets([T]), accumulate=False)
    assert status() == binding.ATTN_OK
    p = torch.exp(s - lse.double().T[..., None])  # [T, 2, rows]
    want = p.sum((0, 1))
    tol = want * 1.01 * (e + 4 * F * most + 4 * F * float(lse.abs().max()) + 2.0 ** -22 + 21 * F)
    got = weights.view(width, page)
    off = (got.double() - want).abs() <= tol
    off[-1, page - 4:] = True  # the last token's position, which the first one does not join, and those behind the end
    assert bool(off.all())
    last = p[1, :, (n - 1) % page].sum()
    assert abs(float(weights.view(-1)[n - 1] - last)) <= float(tol[(n - 1) % page]) and not bool(weights.view(-1)[n:].any())
    # the cut
    cache.table[0, :2] = torch.tensor([1, 2], **i)
    cache.refs.copy_(torch.tensor([width - 2, 1, 1], **i))
    sinks, heavy, recent = 3, 5000, 90
    keep = sinks + heavy + recent
    w = weights.view(-1)
    w.uniform_(generator=g)
    middle = w[sinks:n - recent]
    border = torch.topk(middle, heavy).values[-1]
    above, equal = (middle > border).nonzero()[:, 0], (middle == border).nonzero()[:, 0]
    best = torch.cat([above, equal[:heavy - above.numel()]]).sort().values + sinks
    src = torch.cat([torch.arange(sinks, device="cuda"), best, torch.arange(n - recent, n, device="cuda")])
    at = cache.table[0].long()[src // page]
    want = [x[0, at, 0, src % page] for x in (cache.k, cache.v)] + [w[src]]
    binding.kv_evict(cache, None, weights, sinks=sinks, heavy=heavy, recent=recent)
    assert status() == binding.ATTN_OK
    k, v = gather(cache, 0)
    for a, b in zip(want, (k[:, 0], v[:, 0], w[:keep])):
        assert a.shape == b.shape and torch.equal(a, b)
    assert not bool(w[keep:n].any()) and cache.lens.tolist() == [keep]
    assert cache.refs.tolist() == [0, 1, 1] and bool((cache.table[0, 2:] == -1).all())
