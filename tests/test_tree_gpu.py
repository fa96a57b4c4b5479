"""attn_fwd_tree: draft trees and decoding steps over a paged cache, against 64-bit attention
of each sequence by itself."""
import math
import random

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import DT, close, offsets, plain
from paged_util import build, gather

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return binding.attn_last_device_error(torch.cuda.current_stream())


def trees(sizes, seed, chain=False):
    rng = random.Random(seed)
    return [[t - 1 if chain else (-1 if t == 0 else rng.randint(-1, t - 1)) for t in range(T)] for T in sizes]


def sees(parents, n):
    T = len(parents)
    see = torch.ones(T, n, dtype=torch.bool)
    see[:, n - T:] = False
    for t in range(T):
        u = t
        while u >= 0:
            see[t, n - T + u] = True
            u = parents[u]
    return see


def queries(total, Hq, D, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((total, Hq, D), generator=g, device="cuda") * std).to(DT[dtype])


def check(q, cache, o, lse, rows, par, dtype, scale, layer=0, heads=None):
    Hq, G = q.shape[1], q.shape[1] // cache.Hkv
    a = 0
    for i, (s, p) in enumerate(zip(rows, par)):
        T = len(p)
        if T == 0:
            continue
        k, v = gather(cache, s, layer)
        see = sees(p, k.shape[0])
        for h in range(Hq) if heads is None else heads:
            ro, rl, to, tl = plain(q[a:a + T, h], k[:, h // G], v[:, h // G], see, scale, dtype, pieces=152)
            close(o[a:a + T, h], ro, to, f"O of entry {i}, head {h}")
            close(lse[h, a:a + T], rl, tl, f"LSE of entry {i}, head {h}")
        a += T


CASES = [
    # positions before the tree, tree sizes, Hq, Hkv, D, dtype, page
    ([0], [1], 1, 1, 64, "f16", 16),
    ([0, 5], [1, 2], 2, 1, 128, "bf16", 16),
    ([300], [8], 16, 8, 64, "f16", 16),
    ([127, 128, 129, 1], [1, 1, 1, 1], 8, 2, 128, "bf16", 32),
    ([1000, 0, 64, 700, 255], [26, 64, 0, 1, 33], 8, 2, 128, "bf16", 64),
    ([500, 130], [128, 127], 4, 1, 128, "f16", 128),
    ([500, 130, 77], [100, 65, 64], 6, 2, 64, "bf16", 256),
    ([250, 260, 383, 90], [6, 60, 17, 38], 5, 1, 128, "f16", 16),
    ([2000], [3], 32, 1, 64, "bf16", 64),
    ([40, 3], [2, 9], 128, 1, 64, "f16", 16),
    ([1500, 900], [5, 4], 3, 3, 128, "bf16", 1024),
    ([30 + 17 * i for i in range(70)], [1 + i % 4 for i in range(70)], 2, 1, 64, "bf16", 16),
    ([(7 * i) % 50 for i in range(700)], [1] * 700, 2, 2, 64, "f16", 16),
    ([(7 * i) % 20 for i in range(2300)], [1 + (i % 7 == 0) for i in range(2300)], 2, 1, 64, "f16", 16),
]


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}seqs{sum(c[0])}-{sum(c[1])}-" + "-".join(map(str, c[2:])))
def test_trees(case, chain):
    ctx, T, Hq, Hkv, D, dtype, page = case
    lens = [a + b for a, b in zip(ctx, T)]
    cache = build(lens, page, Hkv, D, dtype, seed=len(ctx))
    par = trees(T, 5, chain)
    q = queries(sum(T), Hq, D, dtype, 7)
    given = None if chain else i32([x for p in par for x in p])
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=given)
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, range(len(ctx)), par, dtype, 1 / math.sqrt(D), heads=None if len(ctx) < 50 else [0])


@pytest.mark.parametrize("Hq,Hkv,D,dtype,T", [(32, 8, 128, "bf16", [128, 100, 0, 37, 1]), (24, 8, 64, "f16", [90, 128, 1, 64, 0]),
                                              (32, 1, 128, "f16", [128, 64, 2, 7, 1])])
def test_many_cut_rows(Hq, Hkv, D, dtype, T):
    """More output rows than the merge takes one by one: it goes over the CTAs' pieces."""
    ctx = [3000, 9001, 500, 0, 7777]
    cache = build([a + b for a, b in zip(ctx, T)], 64, Hkv, D, dtype, seed=48)
    par = trees(T, 49)
    q = queries(sum(T) + 3, Hq, D, dtype, 50)
    out = torch.full_like(q, 7)
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=i32([x for p in par for x in p] + [-1] * 3), out=out)
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, range(5), par, dtype, 1 / math.sqrt(D), heads=[0, Hq // 2, Hq - 1])
    assert bool((o[-3:] == 7).all())


@pytest.mark.parametrize("Hq,Hkv,D,dtype,ctx,T", [
    (16, 8, 128, "bf16", [20000, 300], [128, 60]),
    (32, 8, 128, "bf16", [20001, 9000, 40], [128, 90, 33]),
    (32, 4, 64, "f16", [70000, 1000], [50, 128]),
    (24, 8, 128, "f16", [30000, 0, 12345], [43, 0, 100]),
    (64, 1, 128, "bf16", [20010], [30])])
def test_trees_of_several_row_tiles_over_long_contexts(Hq, Hkv, D, dtype, ctx, T):
    """Several row tiles, each cut over many CTAs, merged by rows and by CTAs."""
    cache = build([a + b for a, b in zip(ctx, T)], 64, Hkv, D, dtype, seed=51)
    par = trees(T, 52)
    q = queries(sum(T), Hq, D, dtype, 53)
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=i32([x for p in par for x in p]))
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, range(len(T)), par, dtype, 1 / math.sqrt(D), heads=[0, Hq // 2 + 1, Hq - 1])


def test_wide_table_of_few_positions():
    """A table for 8 million positions and 128 row tiles a tree: the call goes in launches of few
    sequences, whose weights fit in 32 bits whatever the lengths are."""
    cache = build([5, 130, 64, 200], 64, 1, 64, "f16", width=1 << 17, seed=46)
    rows = [(3 * i) % 4 for i in range(300)]
    q = queries(300, 128, 64, "f16", 47)
    o, lse = binding.attention_tree(q, cache, offsets([1] * 300), seqs=i32(rows))
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, rows, [[-1]] * 300, "f16", 1 / 8, heads=[0, 127])


def test_large_scores_layers_chosen_rows_and_strides():
    """Rows close to one-hot, the second layer, rows of the table in another order and one of
    them twice, queries cut from a projection, an output with strides of its own."""
    ctx, T = [700, 90, 400, 1300], [9, 1, 30, 4]
    cache = build([a + b for a, b in zip(ctx, T)], 32, 2, 128, "bf16", n_layers=2, seed=3)
    rows = [3, 0, 2, 3]
    sizes = [T[s] for s in rows]
    par = trees(sizes, 11)
    x = queries(sum(sizes), 12, 128, "bf16", 9, std=4.0)
    q = x[:, :8]
    wide = torch.zeros((sum(sizes), 10, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((8, sum(sizes)), device="cuda")
    binding.attention_tree(q, cache, offsets(sizes), seqs=i32(rows), parents=i32([y for p in par for y in p]), layer=1,
                           out=wide[:, 1:9], lse_out=lse)
    assert status() == binding.ATTN_OK
    check(q, cache, wide[:, 1:9], lse, rows, par, "bf16", 1 / math.sqrt(128), layer=1)
    assert bool((wide[:, 0] == 0).all()) and bool((wide[:, 9] == 0).all())


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "f16")])
def test_long_contexts_of_different_lengths(D, dtype):
    """Units cut over many CTAs beside short ones."""
    ctx, T = [20011, 3, 130, 7000], [7, 20, 1, 64]
    cache = build([a + b for a, b in zip(ctx, T)], 64, 2, D, dtype, seed=8)
    par = trees(T, 2)
    q = queries(sum(T), 8, D, dtype, 10)
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=i32([x for p in par for x in p]))
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, range(4), par, dtype, 1 / math.sqrt(D), heads=[0, 5])


def test_decoding_step_agrees_with_attn_fwd_decode():
    """One token per sequence over equal lengths: the contiguous cache's decode call on the same
    values, within both calls' bounds."""
    B, N, Hq, Hkv, D = 3, 2111, 8, 2, 128
    cache = build([N] * B, 64, Hkv, D, "bf16", seed=12)
    q = queries(B, Hq, D, "bf16", 13)
    o, lse = binding.attention_tree(q, cache, offsets([1] * B))
    kv = [torch.stack(x).transpose(1, 2).contiguous() for x in zip(*(gather(cache, s) for s in range(B)))]
    o2, lse2 = binding.attention_decode(q.view(B, Hq, 1, D), *kv)
    amax = float(kv[1].abs().max())
    # both: u (|O| + A) and A <= max |v|; here |O| and A stay below 1/4 of it (2111 keys)
    assert float((o.float() - o2.view(B, Hq, D).float()).abs().max()) <= 2 * 2.0 ** -8 * 2 * amax / 4
    assert float((lse - lse2.view(B, Hq).t()).abs().max()) <= 2.0 ** -12


def test_what_lies_outside_a_sequence_stays_out():
    """NaN in the rows of the last page behind the sequence and in every other page; table
    entries behind the sequence are -1 or name NaN pages; rows behind the last tree are left."""
    ctx, T, page = [100, 250, 0], [5, 9, 2], 32
    lens = [a + b for a, b in zip(ctx, T)]
    ok = build(lens, page, 2, 128, "bf16", seed=14)
    k, v = torch.full_like(ok.k, math.nan), torch.full_like(ok.v, math.inf)
    for s, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        at = ok.table[s].long()[pos // page]
        k[0, at, :, pos % page] = ok.k[0, at, :, pos % page]
        v[0, at, :, pos % page] = ok.v[0, at, :, pos % page]
    cache = binding.KVPages(k, v, ok.table, ok.lens, ok.refs)
    cache.table[1, -(-lens[1] // page):] = int((ok.refs == 0).nonzero()[0])
    par = trees(T, 3)
    total = sum(T)
    q = queries(total + 6, 8, 128, "bf16", 15)
    q[total:] = math.nan
    o = torch.full_like(q, 7.0)
    lse = torch.full((8, total + 6), 8.0, device="cuda")
    p = i32([x for t in par for x in t] + [99] * 6)
    binding.attention_tree(q, cache, offsets(T), parents=p, out=o, lse_out=lse)
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, range(3), par, "bf16", 1 / math.sqrt(128))
    assert bool((o[total:] == 7).all()) and bool((lse[:, total:] == 8).all())


@pytest.mark.parametrize("base", [200, 250, 128])
def test_non_finite_values_reach_the_tokens_that_see_them(base):
    T, D = 20, 128
    cache = build([base + T], 64, 2, D, "bf16", seed=16)
    par = trees([T], 21)

    def at(pos):
        return int(cache.table[0, pos // 64]), pos % 64

    for node, col, x in ((3, 0, math.inf), (3, 7, math.nan), (8, 127, -math.inf), (15, 64, math.inf)):
        p, r = at(base + node)
        cache.v[0, p, :, r, col] = x
    q = queries(T, 4, D, "bf16", 17)
    o, lse = binding.attention_tree(q, cache, offsets([T]), parents=i32(par[0]))
    check(q, cache, o, lse, [0], par, "bf16", 1 / math.sqrt(D))
    # a NaN key reaches the tokens that see it only
    p, r = at(base + 10)
    cache.v[0] = cache.v[0].nan_to_num(0, 0, 0)
    cache.k[0, p, :, r] = math.nan
    o, lse = binding.attention_tree(q, cache, offsets([T]), parents=i32(par[0]))
    hit = sees(par[0], base + T)[:, base + 10]
    assert bool(torch.isnan(o[hit.cuda()]).all()) and bool(torch.isfinite(o[~hit.cuda()]).all())
    assert bool(torch.isnan(lse[:, hit.cuda()]).all())


def test_bad_state_is_reported_and_stays_inside():
    """Page indexes out of range or missing, sequences out of range, trees longer than the
    sequence, offsets past the queries: reported; the other sequences are right."""
    ctx, T = [300, 200, 100], [4, 4, 4]
    cache = build([304, 204, 104], 32, 2, 64, "f16", seed=18)
    q = queries(12, 4, 64, "f16", 19)
    par = trees(T, 4)
    p = i32([x for t in par for x in t])
    good = cache.table.clone()
    for wrong in (-1, 10 ** 6, cache.n_pages):
        cache.table[1, 2] = wrong
        o, lse = binding.attention_tree(q, cache, offsets(T), parents=p)
        assert status() == binding.ATTN_ERR_PAGE
        cache.table.copy_(good)
        check(q[:4], cache, o[:4], lse[:, :4], [0], par[:1], "f16", 1 / 8)
        check(q[8:], cache, o[8:], lse[:, 8:], [2], par[2:], "f16", 1 / 8)
    for seqs, cu in (([0, 99, 2], offsets(T)), ([0, -1, 2], offsets(T)), ([0, 1, 2], i32([0, 4, 8, 400]))):
        o, lse = binding.attention_tree(q, cache, cu, seqs=i32(seqs), parents=p)
        assert status() == binding.ATTN_ERR_SHAPE
        check(q[:4], cache, o[:4], lse[:, :4], [0], par[:1], "f16", 1 / 8)
    cache.lens[1] = 2
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=p)
    assert status() == binding.ATTN_ERR_SHAPE
    cache.lens[1] = 204
    # parents that name no earlier token end the walk
    binding.attention_tree(q, cache, offsets(T), parents=i32([5, 0, 99, -7] * 3))
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=p)
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, [0, 1, 2], par, "f16", 1 / 8)


def test_overlapping_offsets_and_trees_past_the_largest():
    """Offsets that go back and forth over the queries, and one tree of 300 tokens: reported, and
    the next call is right."""
    T = [100]
    cache = build([1000] * 8, 32, 2, 64, "f16", seed=41)
    q = queries(100, 8, 64, "f16", 42)
    binding.attention_tree(q, cache, i32([0, 100, 0, 100, 0, 100, 0, 100, 0]))
    assert status() == binding.ATTN_ERR_SHAPE
    binding.attention_tree(queries(300, 8, 64, "f16", 45), cache, offsets([300]))
    assert status() == binding.ATTN_ERR_SHAPE
    o, lse = binding.attention_tree(q, cache, offsets(T))
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, [0], [list(range(-1, 99))], "f16", 1 / 8)


def test_captured_call_replays_on_new_lengths_trees_and_pages():
    cache = build([600, 600, 600], 32, 2, 128, "bf16", seed=20)
    T = [6, 6, 6]
    q = queries(18, 8, 128, "bf16", 21)
    p = i32([x for t in trees(T, 0) for x in t])
    cu = offsets(T)
    o, lse = torch.zeros_like(q), torch.zeros((8, 18), device="cuda")
    n = binding.attn_fwd_tree_workspace(3, 128)[1]
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    binding.attention_tree(q, cache, cu, parents=p, out=o, lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.attention_tree(q, cache, cu, parents=p, out=o, lse_out=lse, workspace=ws)
    for lens, sizes in (([600, 17, 300], [6, 6, 6]), ([129, 599, 64], [1, 16, 1]), ([5, 600, 1], [5, 0, 1])):
        sizes_cu = offsets(sizes)
        cu.copy_(sizes_cu)
        cache.lens.copy_(i32(lens))
        cache.table.copy_(cache.table.flip(0))
        par = trees(sizes, sum(lens))
        p[:sum(sizes)] = i32([x for t in par for x in t])
        q.copy_(queries(18, 8, 128, "bf16", sum(lens)))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        check(q, cache, o, lse, range(3), par, "bf16", 1 / math.sqrt(128))
    assert status() == binding.ATTN_OK


def test_another_stream_and_same_bits():
    cache = build([5000, 40], 64, 2, 128, "bf16", seed=22)
    q = queries(9, 8, 128, "bf16", 23)
    p = i32([x for t in trees([8, 1], 6) for x in t])
    o1, l1 = binding.attention_tree(q, cache, offsets([8, 1]), parents=p)
    s = torch.cuda.Stream()
    cu = offsets([8, 1])
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = binding.attention_tree(q, cache, cu, parents=p, stream=s)
    s.synchronize()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_calls_at_once_on_two_streams():
    """Tree and packed calls on two streams over one cache, each with outputs (and a workspace) of
    its own: the bits of the calls one after another."""
    cache = build([9000, 300, 4000], 64, 2, 128, "bf16", seed=27)
    par = trees([20, 3, 9], 6)
    p = i32([x for t in par for x in t])
    cu, lens = offsets([20, 3, 9]), offsets([700, 40, 300])
    qs = [queries(32, 8, 128, "bf16", 28 + i) for i in range(2)]
    x = [queries(1040, 8, 128, "bf16", 38 + i) for i in range(2)]
    want = [binding.attention_tree(q, cache, cu, parents=p) for q in qs]
    packed = [binding.attention_varlen(y, y[:, :2], y[:, 2:4], lens) for y in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(binding.attention_tree(qs[i], cache, cu, parents=p, stream=s) +
                          binding.attention_varlen(x[i], x[i][:, :2], x[i][:, 2:4], lens,
                                                   stream=s.cuda_stream if i else s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l, po, pl in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
            assert torch.equal(po, packed[i][0]) and torch.equal(pl, packed[i][1])
    assert status() == binding.ATTN_OK


def test_stream_handles():
    """The same bits with the stream as an object, as its handle and as the default stream's."""
    cache = build([3000], 64, 2, 128, "bf16", seed=43)
    q, cu = queries(4, 8, 128, "bf16", 44), offsets([4])
    want = binding.attention_tree(q, cache, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        o, l = binding.attention_tree(q, cache, cu, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    assert status() == binding.ATTN_OK


def test_two_captured_steps_replayed_at_once():
    """Two graphs over one cache, captured with workspaces of their own and replayed on two streams."""
    cache = build([5000, 900], 32, 2, 128, "bf16", seed=29)
    q = [queries(9, 8, 128, "bf16", 30 + i) for i in range(2)]
    cu = offsets([8, 1])
    want = [binding.attention_tree(x, cache, cu) for x in q]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.attention_tree(x, cache, cu))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for o, l in outs:
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    assert status() == binding.ATTN_OK


def test_cache_past_32_bits():
    """A sequence whose pages lie past 2^31 elements of the pool."""
    page, Hkv, D = 128, 8, 128
    n_pages = (1 << 31) // (page * Hkv * D) + 12
    k, v = (torch.zeros((1, n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = torch.full((1, 10), -1, dtype=torch.int32, device="cuda")
    table[0, :9] = torch.arange(n_pages - 9, n_pages, dtype=torch.int32, device="cuda")
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[n_pages - 9:] = 1
    k[0, n_pages - 9:].normal_()
    v[0, n_pages - 9:].normal_()
    cache = binding.KVPages(k, v, table, i32([9 * page - 50]), refs)
    par = trees([12], 1)
    q = queries(12, 16, D, "bf16", 24)
    o, lse = binding.attention_tree(q, cache, offsets([12]), parents=i32(par[0]))
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, [0], par, "bf16", 1 / math.sqrt(D), heads=[0, 15])


def test_timeout_is_reported_and_the_next_call_works():
    lib = binding.load()
    cache = build([700], 32, 2, 128, "bf16", seed=25)
    q = queries(5, 8, 128, "bf16", 26)
    par = trees([5], 1)
    p = i32(par[0])
    binding.attention_tree(q, cache, offsets([5]), parents=p)
    torch.cuda.synchronize()
    try:
        lib.attn_test_set_wait_timeout_ns(50_000_000)
        lib.attn_test_inject_stall(1)
        o, lse = binding.attention_tree(q, cache, offsets([5]), parents=p)
        assert status() == binding.ATTN_ERR_TIMEOUT
    finally:
        lib.attn_test_inject_stall(0)
        lib.attn_test_set_wait_timeout_ns(0)
    o, lse = binding.attention_tree(q, cache, offsets([5]), parents=p)
    assert status() == binding.ATTN_OK
    check(q, cache, o, lse, [0], par, "bf16", 1 / math.sqrt(128))


def test_a_serving_loop():
    """Prompts of different lengths through attn_fwd_varlen, their keys and values into pages,
    draft trees verified over them, the accepted path kept, a fork, a free and a compaction in
    between: each step's attention against the 64-bit sum over what the host says is cached."""
    Hq, Hkv, D, page, dtype = 4, 2, 128, 16, "bf16"
    g = torch.Generator(device="cuda")
    g.manual_seed(31)

    def rows(n, heads):
        return torch.randn((n, heads, D), generator=g, device="cuda").to(torch.bfloat16)

    cache = binding.KVPages.empty(1, 80, Hkv, page, D, 6, 16, torch.bfloat16)
    cache.k.fill_(math.nan)
    cache.v.fill_(math.nan)
    lens = [70, 1, 129]
    q, k, v = rows(200, Hq), rows(200, Hkv), rows(200, Hkv)
    cu = offsets(lens)
    o, lse = binding.attention_varlen(q, k, v, cu)
    binding.kv_extend(cache, i32(lens), i32([0, 1, 2]))
    binding.kv_append(cache, k, v, cu, i32([0, 1, 2]))
    held = {s: (k[a:a + n], v[a:a + n]) for s, a, n in ((0, 0, 70), (1, 70, 1), (2, 71, 129))}
    for s, (a, n) in {0: (0, 70), 1: (70, 1), 2: (71, 129)}.items():
        ro, rl, to, tl = plain(q[a:a + n, 3], held[s][0][:, 1], held[s][1][:, 1],
                               torch.ones(n, n, dtype=torch.bool).tril(), D ** -0.5, dtype)
        close(o[a:a + n, 3], ro, to, "prompt")
    live = [0, 1, 2]
    rng = random.Random(4)
    for step in range(6):
        if step == 2:
            binding.kv_fork(cache, i32([2, 0]), i32([4, 5]))
            held |= {4: held[2], 5: held[0]}
            live += [4, 5]
        if step == 3:
            binding.kv_free(cache, i32([0, 2]))
            live = [1, 4, 5]
        if step == 4:
            binding.kv_compact(cache)
        T = [rng.randint(1, 12) for _ in live]
        par = trees(T, step)
        cu, ids, p = offsets(T), i32(live), i32([x for t in par for x in t])
        q, k, v = rows(sum(T), Hq), rows(sum(T), Hkv), rows(sum(T), Hkv)
        binding.kv_extend(cache, i32(T), ids)
        binding.kv_append(cache, k, v, cu, ids)
        o, lse = binding.attention_tree(q, cache, cu, seqs=ids, parents=p)
        paths, a = [], 0
        for s, t, pp in zip(live, T, par):
            kk, vv = (torch.cat([x, y[a:a + t]]) for x, y in zip(held[s], (k, v)))
            for h in (0, 3):
                ro, rl, to, tl = plain(q[a:a + t, h], kk[:, h // 2], vv[:, h // 2], sees(pp, kk.shape[0]), D ** -0.5, dtype,
                                       pieces=152)
                close(o[a:a + t, h], ro, to, f"step {step}, sequence {s}")
                close(lse[h, a:a + t], rl, tl, f"step {step}, sequence {s}")
            u, path = rng.randrange(t), []
            while u >= 0:
                path.insert(0, u)
                u = pp[u]
            paths.append(path)
            n = held[s][0].shape[0]
            held[s] = tuple(torch.cat([x, y[a:a + t][path]]) for x, y in zip(held[s], (k, v)))
            assert held[s][0].shape[0] == n + len(path)
            a += t
        w = max(map(len, paths))
        binding.kv_accept(cache, cu, i32([x + [-1] * (w - len(x)) for x in paths]), i32(list(map(len, paths))), ids)
        assert cache.lens[ids.long()].tolist() == [held[s][0].shape[0] for s in live]
    assert status() == binding.ATTN_OK
