"""attn_fwd_varlen_window and attn_fwd_tree_window: attention with a sliding window whose first
keys stay visible, against 64-bit attention over the keys that the definition names.  The bounds
are those of the calls without a window (packed_util): the same roundings over fewer keys."""
import math

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import DT, close, offsets, plain
from paged_util import build, gather
from test_tree_gpu import i32, queries, status, trees
from test_varlen_gpu import make

pytestmark = pytest.mark.gpu


def band(nq, nk, window, sinks):
    """Row i stands at position i + nk - nq."""
    p = torch.arange(nk - nq, nk)[:, None]
    j = torch.arange(nk)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def check(q, k, v, o, lse, lens, lens_k, dtype, scale, window, sinks):
    Hq, G = q.shape[1], q.shape[1] // k.shape[1]
    a = b = 0
    for s, (nq, nk) in enumerate(zip(lens, lens_k)):
        see = band(nq, nk, window, sinks)
        for h in range(Hq):
            ro, rl, to, tl = plain(q[a:a + nq, h], k[b:b + nk, h // G], v[b:b + nk, h // G], see, scale, dtype)
            close(o[a:a + nq, h], ro, to, f"O of sequence {s}, head {h}")
            if lse is not None:
                close(lse[h, a:a + nq], rl, tl, f"LSE of sequence {s}, head {h}")
        a, b = a + nq, b + nk


PROMPTS = [
    # lens, window, sinks, Hq, Hkv, D, dtype, layout, std of q, k, v
    ([1], 1, 0, 1, 1, 64, "f16", "packed", 1.0),
    ([5], 2, 1, 2, 1, 128, "bf16", "packed", 1.0),
    ([200], 64, 4, 2, 1, 64, "f16", "packed", 1.0),
    ([129, 1, 0, 255, 256, 257], 1, 0, 4, 2, 128, "bf16", "packed", 1.0),
    ([129, 1, 0, 255, 256, 257], 1, 3, 3, 1, 64, "f16", "fused", 1.0),
    ([129, 1, 0, 255, 256, 257], 100, 0, 4, 2, 64, "f16", "fused", 1.0),
    ([300, 700, 1000], 127, 1, 4, 2, 128, "bf16", "packed", 1.0),
    ([300, 700, 1000], 128, 128, 4, 2, 128, "bf16", "heads", 1.0),
    ([300, 700, 1000], 129, 129, 3, 3, 128, "f16", "packed", 1.0),
    ([1500, 700], 256, 300, 3, 1, 64, "bf16", "packed", 1.0),
    ([1500, 700], 255, 127, 2, 1, 128, "f16", "fused", 2.0),
    ([1500, 2], 640, 5, 5, 5, 64, "f16", "packed", 1.0),
    ([2100], 900, 0, 2, 1, 128, "bf16", "packed", 4.0),
    ([900, 30], 5000, 2, 4, 2, 128, "bf16", "packed", 1.0),     # longer than every sequence
    ([900, 30], 20, 5000, 4, 2, 128, "bf16", "packed", 1.0),    # all keys are first ones
    ([900, 400], 20, 890, 4, 2, 128, "bf16", "packed", 1.0),
    ([1 + (7 * i) % 11 for i in range(200)], 3, 1, 2, 1, 64, "bf16", "packed", 1.0),
    ([(5 * i) % 3 for i in range(2500)], 1, 0, 1, 1, 64, "f16", "packed", 1.0),
]


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-" + "-".join(map(str, c[1:])))
def test_packed_prompts(case):
    lens, window, sinks, Hq, Hkv, D, dtype, layout, std = case
    q, k, v = make(sum(lens), Hq, Hkv, D, dtype, layout, std, seed=len(lens) + Hq + D)
    o, lse = binding.attention_varlen(q, k, v, offsets(lens), window=window, sinks=sinks)
    assert status() == binding.ATTN_OK
    check(q, k, v, o, lse, lens, lens, dtype, 1 / math.sqrt(D), window, sinks)


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (200, 140), (1 << 40, 0)])
def test_chunks_over_longer_keys(Hq, Hkv, window, sinks):
    """The queries are the last positions of longer keys; more queries than keys (rows that see
    nothing), no keys, no queries."""
    lens_q = [64, 1, 130, 200, 300, 5, 0, 140, 257]
    lens_k = [720, 1013, 131, 200, 100, 0, 40, 1, 900]
    q, k, v = make(sum(lens_q), Hq, Hkv, 128, "bf16", seed=3, total_k=sum(lens_k))
    o, lse = binding.attention_varlen(q, k, v, offsets(lens_q), offsets(lens_k), scale=0.11, window=window, sinks=sinks)
    assert status() == binding.ATTN_OK
    check(q, k, v, o, lse, lens_q, lens_k, "bf16", 0.11, window, sinks)


def test_a_window_without_effect_gives_the_same_bits():
    q, k, v = make(700, 4, 2, 128, "bf16", seed=8)
    cu = offsets([500, 200])
    o, lse = binding.attention_varlen(q, k, v, cu)
    o2, lse2 = binding.attention_varlen(q, k, v, cu, window=700, sinks=3)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 128, "bf16"), (3, 1, 64, "f16")])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_non_finite_values_reach_the_rows_that_see_them(Hq, Hkv, D, dtype, bad):
    """Keys on both borders of many windows, among the first keys and behind them; keys that no
    row of a block sees; padding rows behind the last sequence and another sequence, all NaN."""
    lens, window, sinks, pad = [1100, 200, 130], 300, 10, 70
    total = sum(lens)
    q, k, v = make(total + pad, Hq, Hkv, D, dtype, seed=21)
    v[[3, 9, 10, 127, 128, 300, 555, 700, 1099], :, 5] = bad
    k[[10, 400], 0] = bad  # a key's scores: NaN or infinite in the rows that see it
    for x in (q, k, v):
        x[1100:1300] = math.nan
        x[total:] = math.nan
    out, lse_out = torch.full_like(q, 7.0), torch.full((Hq, total + pad), 8.0, device="cuda")
    o, lse = binding.attention_varlen(q, k, v, offsets(lens), window=window, sinks=sinks, out=out, lse_out=lse_out)
    assert bool((o[total:] == 7).all()) and bool((lse[:, total:] == 8).all())
    assert bool(torch.isnan(o[1100:1300]).all())
    see = band(1100, 1100, window, sinks)
    hit = see[:, [10, 400]].any(1)
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        clean = ~hit if kv == 0 else torch.ones(1100, dtype=torch.bool)
        kk = k[:1100, kv].clone()
        kk[[10, 400]] = 0.0
        vv = v[:1100, kv]
        ro, rl, to, tl = plain(q[:1100, h], kk if kv == 0 else k[:1100, kv], vv, see, 1 / math.sqrt(D), dtype)
        close(o[:1100, h].cpu()[clean], ro[clean], to[clean].nan_to_num(0, 0, 0), f"head {h}")
        close(lse[h, :1100].cpu()[clean], rl[clean], tl[clean], f"LSE of head {h}")
    check(q[1300:total], k[1300:total], v[1300:total], o[1300:total], lse[:, 1300:total], [130], [130], dtype,
          1 / math.sqrt(D), window, sinks)


def sees(parents, n, window, sinks):
    """What token t's own sequence (positions before the tree, its ancestors, itself) shows it."""
    T = len(parents)
    see = torch.zeros(T, n, dtype=torch.bool)
    for t in range(T):
        path, u = [], t
        while u >= 0:
            path.append(n - T + u)
            u = parents[u]
        path = list(range(n - T)) + path[::-1]
        see[t, path[-window:]] = True
        see[t, path[:sinks]] = True
    return see


def check_trees(q, cache, o, lse, rows, par, dtype, scale, window, sinks, layer=0, heads=None):
    Hq, G = q.shape[1], q.shape[1] // cache.Hkv
    a = 0
    for i, (s, p) in enumerate(zip(rows, par)):
        T = len(p)
        if T == 0:
            continue
        k, v = gather(cache, s, layer)
        see = sees(p, k.shape[0], window, sinks)
        for h in range(Hq) if heads is None else heads:
            ro, rl, to, tl = plain(q[a:a + T, h], k[:, h // G], v[:, h // G], see, scale, dtype, pieces=152)
            close(o[a:a + T, h], ro, to, f"O of entry {i}, head {h}")
            close(lse[h, a:a + T], rl, tl, f"LSE of entry {i}, head {h}")
        a += T


TREES = [
    # positions before the tree, tree sizes, window, sinks, Hq, Hkv, D, dtype, page
    ([0], [1], 1, 0, 1, 1, 64, "f16", 16),
    ([0, 5], [1, 2], 1, 1, 2, 1, 128, "bf16", 16),
    ([300], [8], 64, 4, 16, 8, 64, "f16", 16),
    ([127, 128, 129, 1, 900], [1, 1, 1, 1, 1], 128, 4, 8, 2, 128, "bf16", 32),
    ([1000, 0, 64, 700, 255], [26, 64, 0, 1, 33], 20, 1, 8, 2, 128, "bf16", 64),
    ([1000, 0, 64, 700, 255], [26, 64, 0, 1, 33], 300, 130, 8, 2, 128, "bf16", 64),
    ([500, 130], [128, 127], 3, 0, 4, 1, 128, "f16", 128),
    ([500, 130], [128, 127], 100, 5, 4, 1, 128, "f16", 128),
    ([1500, 130, 977], [100, 65, 64], 129, 300, 6, 2, 64, "bf16", 256),
    ([250, 260, 383, 90], [6, 60, 17, 38], 40, 100, 5, 1, 128, "f16", 16),
    ([5000], [3], 513, 2, 32, 1, 64, "bf16", 64),
    ([40, 3], [2, 9], 4, 2, 128, 1, 64, "f16", 16),
    ([3500, 2900], [5, 4], 700, 600, 3, 3, 128, "bf16", 1024),
    ([9000, 5], [1, 1], 1100, 128, 8, 2, 128, "bf16", 4096),
    ([60, 20], [70, 60], 90, 70, 8, 2, 64, "f16", 16),  # first keys that reach into the trees
    ([30 + 37 * i for i in range(70)], [1 + i % 4 for i in range(70)], 200, 4, 2, 1, 64, "bf16", 16),
    ([(7 * i) % 500 for i in range(700)], [1] * 700, 60, 1, 2, 2, 64, "f16", 16),
]


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("case", TREES, ids=lambda c: f"{len(c[0])}seqs{sum(c[0])}-{sum(c[1])}-" + "-".join(map(str, c[2:])))
def test_trees_over_pages(case, chain):
    ctx, T, window, sinks, Hq, Hkv, D, dtype, page = case
    cache = build([a + b for a, b in zip(ctx, T)], page, Hkv, D, dtype, seed=len(ctx))
    par = trees(T, 5, chain)
    q = queries(sum(T), Hq, D, dtype, 7)
    given = None if chain else i32([x for p in par for x in p])
    o, lse = binding.attention_tree(q, cache, offsets(T), parents=given, window=window, sinks=sinks)
    assert status() == binding.ATTN_OK
    check_trees(q, cache, o, lse, range(len(ctx)), par, dtype, 1 / math.sqrt(D), window, sinks,
                heads=None if len(ctx) < 50 else [0])


@pytest.mark.parametrize("Hq,Hkv,D,dtype,page", [(32, 8, 128, "bf16", 64), (24, 8, 64, "f16", 16)])
def test_long_windows_cut_over_many_ctas(Hq, Hkv, D, dtype, page):
    """Units cut into pieces, merged by rows and (the second call) by CTAs; a table order and a
    sequence named twice."""
    ctx = [30000, 9001, 500, 0, 17777]
    for T, rows in (([1, 7, 20, 1, 3], [4, 1, 0, 3, 4]), ([100, 128, 0, 37, 100], [0, 1, 2, 3, 0])):
        most = [max([t for t, r in zip(T, rows) if r == s], default=0) for s in range(5)]
        cache = build([a + b for a, b in zip(ctx, most)], page, Hkv, D, dtype, seed=48)
        par = trees(T, 49)
        q = queries(sum(T), Hq, D, dtype, 50)
        o, lse = binding.attention_tree(q, cache, offsets(T), seqs=i32(rows), parents=i32([x for p in par for x in p]),
                                        window=7000, sinks=150)
        assert status() == binding.ATTN_OK
        check_trees(q, cache, o, lse, rows, par, dtype, 1 / math.sqrt(D), 7000, 150, heads=[0, Hq - 1])


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_outside_the_window_stay_out(T, bad):
    """Positions between the first keys and the window hold NaN or infinities, as do the rows
    behind the end and every other page; pages that nobody sees are missing from the table."""
    ctx, window, sinks, page = [1000, 450], 200, 20, 16
    lens = [c + T for c in ctx]
    ok = build(lens, page, 2, 128, "bf16", seed=14)
    k, v = torch.full_like(ok.k, bad), torch.full_like(ok.v, bad)
    par = [[-1] + list(range(T - 1))] * 2
    for s, n in enumerate(lens):
        pos = torch.cat([torch.arange(sinks), torch.arange(ctx[s] - window + 1, n)]).cuda()
        at = ok.table[s].long()[pos // page]
        k[0, at, :, pos % page] = ok.k[0, at, :, pos % page]
        v[0, at, :, pos % page] = ok.v[0, at, :, pos % page]
    table = ok.table.clone()
    table[0, 8:48] = -1  # positions 128 .. 767: the window begins in 801, in the run from 768 on
    cache = binding.KVPages(k, v, table, ok.lens, ok.refs)
    q = queries(2 * T, 8, 128, "bf16", 15)
    o, lse = binding.attention_tree(q, cache, offsets([T, T]), window=window, sinks=sinks)
    assert status() == binding.ATTN_OK
    whole = binding.KVPages(ok.k, ok.v, ok.table, ok.lens, ok.refs)
    check_trees(q, whole, o, lse, range(2), par, "bf16", 1 / math.sqrt(128), window, sinks)
    # one within the run is read, and missed
    table[0, 48] = -1
    binding.attention_tree(q, cache, offsets([T, T]), window=window, sinks=sinks)
    assert status() == binding.ATTN_ERR_PAGE


def test_non_finite_values_in_a_window_reach_the_tokens_that_see_them():
    """A tree over a window: values at positions that some tokens see and others do not."""
    ctx, T, window, sinks = 900, 40, 30, 3
    cache = build([ctx + T], 32, 2, 64, "f16", seed=16)
    par = trees([T], 17)[0]
    for j, x in ((2, math.inf), (ctx - 29, math.nan), (ctx - 20, -math.inf), (ctx - 1, math.inf), (ctx + 7, math.nan),
                 (ctx + 20, math.inf), (500, math.nan), (3, math.inf)):
        cache.v[0, int(cache.table[0, j // 32]), :, j % 32, j % 64] = x
    q = queries(T, 4, 64, "f16", 18)
    o, lse = binding.attention_tree(q, cache, offsets([T]), parents=i32(par), window=window, sinks=sinks)
    assert status() == binding.ATTN_OK
    k, v = gather(cache, 0)
    see = sees(par, ctx + T, window, sinks)
    for h in range(4):
        ro, rl, to, tl = plain(q[:, h], k[:, h // 2], v[:, h // 2], see, 1 / 8, "f16")
        close(o[:, h], ro, to.nan_to_num(0, 0, 0), f"head {h}")
        close(lse[h], rl, tl, f"LSE of head {h}")


def test_captured_calls_replay_on_new_lengths():
    """Both calls in one graph on a side stream, replayed on other offsets, lengths and trees."""
    q, k, v = make(600, 4, 2, 128, "bf16", seed=31)
    cache = build([700, 300], 32, 2, 128, "bf16", seed=32, width=40)
    tq = queries(12, 4, 128, "bf16", 33)
    cu, tcu, par = offsets([400, 200]), offsets([7, 5]), i32([-1] * 12)
    o, lse = torch.empty_like(q), torch.empty((4, 600), device="cuda")
    to, tlse = torch.empty_like(tq), torch.empty((4, 12), device="cuda")
    st, nbytes = binding.attn_fwd_tree_workspace(2, 128)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def step():
        binding.attention_varlen(q, k, v, cu, window=150, sinks=4, out=o, lse_out=lse)
        binding.attention_tree(tq, cache, tcu, parents=par, window=150, sinks=4, out=to, lse_out=tlse, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for lens, T, ctx in (([400, 200], [7, 5], [700, 300]), ([1, 599], [2, 10], [130, 290]), ([300, 0], [12, 0], [512, 9])):
        cu.copy_(offsets(lens))
        tcu.copy_(offsets(T))
        cache.lens.copy_(i32(ctx))
        par_h = trees(T, sum(T) + lens[0])
        par.copy_(i32([x for p in par_h for x in p]))
        graph.replay()
        torch.cuda.synchronize()
        assert status() == binding.ATTN_OK
        n = sum(lens)
        check(q[:n], k[:n], v[:n], o[:n], lse[:, :n], lens, lens, "bf16", 1 / math.sqrt(128), 150, 4)
        check_trees(tq, cache, to, tlse, range(2), par_h, "bf16", 1 / math.sqrt(128), 150, 4)


def test_refusals():
    q, k, v = make(8, 2, 1, 64, "f16")
    cache = build([8], 16, 1, 64, "f16")
    cu = offsets([8])
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(binding.AttnError):
            binding.attention_varlen(q, k, v, cu, window=window, sinks=sinks)
        with pytest.raises(binding.AttnError):
            binding.attention_tree(q, cache, cu, window=window, sinks=sinks)
    with pytest.raises(ValueError):
        binding.attention_varlen(q, k, v, cu, causal=False, window=4)
    with pytest.raises(ValueError):
        binding.attention_varlen(q, k, v, cu, sinks=4)
    with pytest.raises(ValueError):
        binding.attention_tree(q, cache, cu, sinks=4)
    assert status() == binding.ATTN_OK
