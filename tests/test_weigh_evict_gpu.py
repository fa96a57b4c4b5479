"""attn_kv_weigh and attn_kv_evict: the attention weight of cached positions against the formula in
64 bits, and eviction against the same operator written out in Python (equal bits).

Bound of a sum of weights, from the kernel's arithmetic (f = 2^-24): a score is an fp32 sum of D
products, off by e = (D + 2) f scale sum_d |q_d k_d|; its exponent, in natural units, by f |s| for the
scale, 2 f |lse| for the log-sum-exp's product with log2 e and f |s - lse| for the one rounding of
their difference; ex2 is off by 2^-22 of its value.  Within a tile of 128 rows 4 chains of 32 are
added, then 2 sums, then one sum per row tile and the old value: (32 + 2 + tiles + 1) f of the sum."""
import math

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import F, close, offsets
from paged_util import Model, build, gather
from test_tree_gpu import check, i32, queries, status, trees

pytestmark = pytest.mark.gpu


def logsumexps(q, k, T, scale):
    """fp32 [Hq, T] of the last T positions of a sequence (k [n, Hkv, D])."""
    n, G = k.shape[0], q.shape[1] // k.shape[1]
    s = torch.einsum("thd,nhd->htn", q.double(), k.double().repeat_interleave(G, 1)) * scale
    see = torch.ones(T, n, dtype=torch.bool, device=q.device).tril(n - T)
    return torch.logsumexp(s.masked_fill(~see, -math.inf), -1).float()


def weigh_plain(q, lse, k, T, scale):
    """Sums [Hkv, n] in 64 bits and their bounds; q [T, Hq, D], lse [Hq, T]."""
    n, Hkv, D = k.shape
    G = q.shape[1] // Hkv
    q, k, lse = q.double().cpu(), k.double().cpu(), lse.double().cpu()
    see = torch.ones(T, n, dtype=torch.bool).tril(n - T)
    sums, tol = torch.zeros(Hkv, n, dtype=torch.float64), torch.zeros(Hkv, n, dtype=torch.float64)
    tiles = -(-T // (128 // G))
    for h in range(Hkv * G):
        s = q[:, h] @ k[:, h // G].T * scale
        e = (D + 2) * F * (q[:, h].abs() @ k[:, h // G].abs().T) * scale
        l = lse[h][:, None]
        p = torch.where(see, torch.exp(s - l), 0.0)
        d = e + F * s.abs() + 2 * F * l.abs() + F * (s - l).abs() + 2.0 ** -22
        sums[h // G] += p.sum(0)
        tol[h // G] += torch.where(see, p * d * (1 + d), 0.0).sum(0)
    return sums, tol + (35 + tiles) * F * sums + 1e-30


WEIGH = [
    # lengths, tokens, Hq, Hkv, D, dtype, page
    ([1], [1], 1, 1, 64, "f16", 16),
    ([300], [1], 2, 1, 128, "bf16", 16),
    ([257, 256, 255, 1, 600], [1, 1, 1, 1, 1], 8, 2, 128, "bf16", 64),
    ([257, 256, 0, 129, 600], [257, 3, 0, 129, 5], 8, 2, 64, "f16", 32),
    ([700, 130], [700, 1], 4, 2, 128, "bf16", 128),
    ([700, 130], [33, 130], 6, 2, 64, "bf16", 256),
    ([1100], [1100], 3, 1, 128, "f16", 16),
    ([1000, 513], [9, 300], 5, 1, 64, "f16", 1024),
    ([900, 40], [50, 40], 128, 1, 64, "bf16", 64),
    ([900, 40], [2, 1], 24, 1, 128, "f16", 4096),
    ([2000], [64], 32, 8, 128, "bf16", 64),
    ([(7 * i) % 500 + 1 for i in range(150)], [1 + (i % 3 == 0) * ((7 * i) % 500) // 2 for i in range(150)], 2, 2, 64, "bf16", 16),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", WEIGH, ids=lambda c: f"{len(c[0])}seqs{sum(c[0])}-{sum(c[1])}-" + "-".join(map(str, c[2:])))
def test_weights_of_positions(case, accumulate):
    lens, T, Hq, Hkv, D, dtype, page = case
    cache = build(lens, page, Hkv, D, dtype, n_layers=2, seed=len(lens))
    q, scale = queries(sum(T), Hq, D, dtype, 7), 1 / math.sqrt(D)
    lse, a = torch.empty((Hq, sum(T)), device="cuda"), 0
    for s, t in enumerate(T):
        lse[:, a:a + t] = logsumexps(q[a:a + t], gather(cache, s, 1)[0], t, scale)
        a += t
    weights = cache.weights() + 3.0
    weights[1].uniform_(0.0, 2.0)
    old = weights.clone()
    binding.kv_weigh(cache, weights, q, lse, offsets(T), layer=1, accumulate=accumulate)
    assert status() == binding.ATTN_OK
    assert torch.equal(weights[0], old[0])
    again, a = old.clone(), 0
    binding.kv_weigh(cache, again, q, lse, offsets(T), layer=1, accumulate=accumulate)
    assert torch.equal(weights, again)  # one order of the sums
    for s, (n, t) in enumerate(zip(lens, T)):
        got, was = weights[1, s].double().cpu(), old[1, s].double().cpu()
        assert torch.equal(got[:, n if t else 0:], was[:, n if t else 0:])
        if t:
            want, tol = weigh_plain(q[a:a + t], lse[:, a:a + t], gather(cache, s, 1)[0], t, scale)
            if accumulate:
                want[:, :n - t] += was[:, :n - t]
                tol[:, :n - t] += F * want[:, :n - t]
            close(got[:, :n], want, tol, f"sequence {s}")
        a += t


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, "bf16"), (3, 1, 64, "f16")])
def test_weights_leave_out_what_no_pair_joins(Hq, Hkv, D, dtype):
    """Large scores; NaN in rows behind the sequence, in other pages, in a later sequence's queries
    and in a later token's key: no other sum changes.  Queries cut from a projection, chosen rows."""
    lens, T, page, scale = [400, 150, 270], [20, 60, 270], 32, 0.2
    rows = [2, 0, 1]
    ok = build(lens, page, Hkv, D, dtype, seed=3)
    k = torch.full_like(ok.k, math.nan)
    for s, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        at = ok.table[s].long()[pos // page]
        k[0, at, :, pos % page] = ok.k[0, at, :, pos % page]
    cache = binding.KVPages(k, torch.full_like(ok.v, math.nan), ok.table, ok.lens, ok.refs)
    new = [T[s] for s in rows]
    x = queries(sum(new) + 5, Hq + 2, D, dtype, 9, std=3.0)
    q = x[:, 1:Hq + 1]
    q[sum(new):] = math.nan
    lse, a = torch.full((Hq, sum(new) + 5), math.nan, device="cuda"), 0
    for s in rows:
        lse[:, a:a + T[s]] = logsumexps(q[a:a + T[s]], gather(cache, s)[0], T[s], scale)
        a += T[s]
    last = int(ok.table[1, (lens[1] - 1) // page])
    cache.k[0, last, :, (lens[1] - 1) % page] = math.nan  # the last token's key: only that token joins it
    q[sum(new) - 1] = math.nan
    weights = cache.weights()
    binding.kv_weigh(cache, weights, q, lse, offsets(new), seqs=i32(rows), scale=scale)
    assert status() == binding.ATTN_OK
    a = 0
    for s in rows:
        n, t = lens[s], T[s]
        if s != 1:
            want, tol = weigh_plain(q[a:a + t], lse[:, a:a + t], gather(cache, s)[0], t, scale)
            close(weights[0, s, :, :n], want, tol, f"sequence {s}")
        assert bool((weights[0, s, :, n:] == 0).all())
        a += t
    assert bool(torch.isnan(weights[0, 1, :, lens[1] - 1]).all())


def test_weigh_refuses_what_is_out_of_range():
    cache = build([100, 50, 80], 16, 1, 64, "f16")
    q, lse = queries(30, 2, 64, "f16", 1), torch.zeros((2, 30), device="cuda")
    for cu, seqs, bad in (([0, 10, 20, 30], [0, 5, -1], [1, 2]), ([0, 10, 20, 30], [1, 1, 0], [1]),
                          ([0, 10, 5, 30], [0, 1, 2], [1, 2]), ([0, 60, 60, 60], [0, 1, 2], [0, 1, 2])):
        weights = cache.weights() + 1
        binding.kv_weigh(cache, weights, q, lse, i32(cu), seqs=i32(seqs))
        assert status() == binding.ATTN_ERR_SHAPE
        done = {s for i, s in enumerate(seqs) if i not in bad and 0 <= s < 3}
        for s in range(3):
            if s not in done:
                assert bool((weights[0, s] == 1).all())
    cache.lens[1] = 5  # fewer positions than tokens
    weights = cache.weights() + 1
    binding.kv_weigh(cache, weights, q, lse, i32([0, 10, 20]), seqs=i32([0, 1]))
    assert status() == binding.ATTN_ERR_SHAPE
    assert bool((weights[0, 1] == 1).all()) and not bool((weights[0, 0, 0, :100] == 1).any())
    cache.table[0, 3] = -1
    binding.kv_weigh(cache, weights, q, lse, i32([0, 10]), seqs=i32([0]))
    assert status() == binding.ATTN_ERR_PAGE


def test_weigh_over_a_long_list_of_chosen_rows():
    """More entries than are looked through one by one: each row's first entry counts, the others are refused."""
    lens = [1 + (13 * i) % 300 for i in range(90)]
    cache = build(lens, 16, 2, 64, "bf16", seed=41)
    rows = [(7 * i) % 90 for i in range(90)]
    rows[20], rows[70], rows[89], rows[5] = rows[3], rows[69], rows[0], -1
    q, scale = queries(90, 4, 64, "bf16", 42), 1 / 8
    lse = torch.zeros((4, 90), device="cuda")
    for i, s in enumerate(rows):
        lse[:, i:i + 1] = logsumexps(q[i:i + 1], gather(cache, max(s, 0))[0], 1, scale)
    weights = cache.weights() + 1
    binding.kv_weigh(cache, weights, q, lse, offsets([1] * 90), seqs=i32(rows))
    assert status() == binding.ATTN_ERR_SHAPE
    for s in range(90):
        if s not in rows:
            assert bool((weights[0, s] == 1).all())
            continue
        i, n = rows.index(s), lens[s]
        want, tol = weigh_plain(q[i:i + 1], lse[:, i:i + 1], gather(cache, s)[0], 1, scale)
        want[:, :n - 1] += 1
        close(weights[0, s, :, :n], want, tol + F * want, f"row {s}")
        assert bool((weights[0, s, :, n:] == 1).all())


# ---------------------------------------------------------------- eviction
def evict(model, weights, seqs, sinks, heavy, recent):
    """The operator on a host model of the cache, and on its weights (a list of arrays, or None)."""
    keep, page = sinks + heavy + recent, model.page
    for s in seqs:
        n = model.lens[s]
        if n <= keep:
            continue
        layers, _, Hkv = model.k.shape[:3]
        src = {}
        for layer in range(layers):
            for h in range(Hkv):
                order = list(range(sinks, n - recent))
                if heavy:
                    w = [float(x) for x in weights[layer, s, h]]
                    w = [x if x > 0 else 0.0 for x in w]  # NaN and negative ones, too
                    order.sort(key=lambda j: (-w[j], j))
                src[layer, h] = list(range(sinks)) + sorted(order[:heavy]) + list(range(n - recent, n))
        k, v, w = model.k.clone(), model.v.clone(), None if weights is None else weights.clone()
        for (layer, h), at in src.items():
            for d, j in enumerate(at):
                a, b = model.table[s][j // page], model.table[s][d // page]
                model.k[layer, b, h, d % page] = k[layer, a, h, j % page]
                model.v[layer, b, h, d % page] = v[layer, a, h, j % page]
                if w is not None:
                    weights[layer, s, h, d] = w[layer, s, h, j]
            if w is not None:
                weights[layer, s, h, keep:n] = 0.0
        for j in range(-(-keep // page), model.width):
            if model.table[s][j] >= 0:
                model.refs[model.table[s][j]] -= 1
                model.table[s][j] = -1
        model.lens[s] = keep


def same_weights(got, want):
    assert torch.equal(got.cpu().view(torch.int32), want.view(torch.int32))


EVICT = [
    # lengths, sinks, heavy, recent, layers, Hkv, D, dtype, page
    ([5], 1, 1, 1, 1, 1, 64, "f16", 16),
    ([1, 0, 2], 0, 0, 1, 1, 1, 128, "bf16", 16),
    ([100, 64, 63, 65, 300], 4, 30, 30, 2, 2, 64, "f16", 16),
    ([100, 64, 63, 65, 300], 0, 1, 0, 2, 2, 128, "bf16", 32),
    ([100, 64, 63, 65, 300], 20, 0, 33, 1, 3, 128, "bf16", 64),
    ([100, 64, 63, 65, 300], 40, 7, 0, 1, 1, 64, "bf16", 256),
    ([100, 64], 40, 0, 0, 1, 2, 64, "bf16", 16),
    ([100, 64], 0, 0, 0, 1, 2, 64, "bf16", 16),
    ([3000, 2050, 2049], 3, 1500, 500, 1, 2, 64, "f16", 128),
    ([5000, 7000], 17, 4096, 800, 1, 1, 128, "bf16", 64),
    ([5000], 0, 4999, 0, 1, 1, 64, "bf16", 1024),
]


@pytest.mark.parametrize("kind", ["spread", "equal", "few", "odd"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{len(c[0])}seqs{sum(c[0])}-" + "-".join(map(str, c[1:])))
def test_eviction(case, kind):
    lens, sinks, heavy, recent, layers, Hkv, D, dtype, page = case
    cache = build(lens, page, Hkv, D, dtype, n_layers=layers, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    weights = torch.rand(cache.weights().shape, generator=g, device="cuda")
    if kind == "equal":
        weights[:] = 0.25
    elif kind == "few":  # few values, many ties, zeros
        weights = torch.floor(weights * 4) * 1e-3
    elif kind == "odd":
        weights = torch.exp(60 * weights - 45)
        for j, x in enumerate((math.nan, math.inf, -1.0, -0.0, 0.0, 1e-42, -math.inf, 3e38)):
            weights[..., j::37] = x
    model, host = Model(cache), weights.cpu()
    order = list(range(len(lens)))[::-1]
    binding.kv_evict(cache, i32(order), weights, sinks=sinks, heavy=heavy, recent=recent)
    assert status() == binding.ATTN_OK
    evict(model, host, order, sinks, heavy, recent)
    model.same(cache)
    model.consistent()
    same_weights(weights, host)


def test_the_oldest_go_without_weights_and_all_sequences_are_meant():
    cache = build([700, 30, 300, 131], 32, 2, 128, "bf16", n_layers=2, seed=9)
    model = Model(cache)
    binding.kv_evict(cache, sinks=4, recent=127)
    assert status() == binding.ATTN_OK
    evict(model, None, range(4), 4, 0, 127)
    model.same(cache)


def test_shared_pages():
    """A forked sequence: whole shared pages of first positions stay shared, a shared page that would
    be written is refused, and a shared one that is only read is not."""
    cache = build([100, 0, 60], 16, 2, 64, "f16", seed=11, extra_pages=12, width=10)
    binding.kv_fork(cache, i32([0]), i32([1]))
    weights = torch.rand(cache.weights().shape, device="cuda")
    model, host = Model(cache), weights.cpu()
    binding.kv_evict(cache, i32([1, 2]), weights, sinks=32, heavy=3, recent=10)  # writes pages 2: shared
    assert status() == binding.ATTN_ERR_PAGE
    evict(model, host, [2], 32, 3, 10)
    model.same(cache)
    same_weights(weights, host)
    binding.kv_evict(cache, i32([1]), weights, sinks=96, heavy=0, recent=1)  # the last page is its own
    assert status() == binding.ATTN_OK
    evict(model, host, [1], 96, 0, 1)
    model.same(cache)
    # the parent's first page has become its own again, the others are shared: it writes the first only
    cache.table[1, 0] = -1
    cache.refs[int(cache.table[0, 0])] = 1
    model = Model(cache)
    binding.kv_evict(cache, i32([0]), weights, sinks=2, heavy=4, recent=10)
    assert status() == binding.ATTN_OK
    host = host.clone()
    evict(model, host, [0], 2, 4, 10)
    model.same(cache)
    same_weights(weights, host)


def test_eviction_refuses_what_is_wrong():
    cache = build([100, 90, 80, 70], 16, 1, 64, "f16", seed=12)
    weights = torch.rand(cache.weights().shape, device="cuda")
    model, host = Model(cache), weights.cpu()
    with pytest.raises(binding.AttnError):  # more entries than rows
        binding.kv_evict(cache, i32([2, -1, 0, 4, 2]), weights, sinks=1, heavy=8, recent=8)
    binding.kv_evict(cache, i32([4]), weights, sinks=1, heavy=8, recent=8)
    assert status() == binding.ATTN_ERR_SHAPE
    binding.kv_evict(cache, i32([2, -1, 0, 2]), weights, sinks=1, heavy=8, recent=8)  # 2 twice
    assert status() == binding.ATTN_ERR_SHAPE
    evict(model, host, [2, 0], 1, 8, 8)
    model.same(cache)
    same_weights(weights, host)
    cache.table[1, 4] = -1
    cache.lens[3] = 5000
    model = Model(cache)
    binding.kv_evict(cache, i32([1]), weights, sinks=1, heavy=8, recent=8)
    assert status() == binding.ATTN_ERR_PAGE
    binding.kv_evict(cache, i32([3]), weights, sinks=1, heavy=8, recent=8)
    assert status() == binding.ATTN_ERR_SHAPE
    model.same(cache)
    same_weights(weights, host)
    with pytest.raises(binding.AttnError):
        binding.kv_evict(cache, i32([1]), None, heavy=1)
    with pytest.raises(binding.AttnError):
        binding.kv_evict(cache, i32([1]), weights, sinks=-1)
    with pytest.raises(ValueError):
        binding.kv_evict(cache, i32([1]), weights[:, :, :, 1:], heavy=1)
    with pytest.raises(ValueError):
        binding.kv_weigh(cache, weights.half(), queries(3, 2, 64, "f16", 1), torch.zeros((2, 3), device="cuda"), offsets([3]))


def test_a_bounded_cache_as_it_is_used():
    """Prompts through the window and through all keys, their keys into pages, their weights; then steps
    of single tokens and drafted trees, weighed, cut back again and again; one step in a graph."""
    Hq, Hkv, D, dtype, page, scale = 8, 2, 128, "bf16", 16, 1 / math.sqrt(128)
    lens, keeps = [200, 90, 300], dict(sinks=4, heavy=40, recent=36)
    cache = binding.KVPages.empty(1, 80, Hkv, page, D, 4, 40, torch.bfloat16)
    weights, rows = cache.weights(), i32([0, 1, 2])
    x = queries(sum(lens), Hq + 2 * Hkv, D, dtype, 21)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu = offsets(lens)
    binding.kv_extend(cache, i32(lens), seqs=rows)
    binding.kv_append(cache, k, v, cu, seqs=rows)
    o, lse = binding.attention_varlen(q, k, v, cu)
    binding.kv_weigh(cache, weights, q, lse, cu, seqs=rows, accumulate=False)
    a = 0
    for s, n in enumerate(lens):
        want, tol = weigh_plain(q[a:a + n], lse[:, a:a + n], k[a:a + n], n, scale)
        close(weights[0, s, :, :n], want, tol, f"prompt {s}")
        # each row pays 1 in all, and there are 4 heads to a kv head
        assert float((weights[0, s].sum(-1) - 4 * n).abs().max()) < 4 * n * 2.0 ** -12
        a += n
    model = Model(cache)
    host = weights.cpu()

    def cut():
        nonlocal host
        host = weights.cpu()
        model.__init__(cache)
        binding.kv_evict(cache, rows, weights, **keeps)
        evict(model, host, range(3), **keeps)
        assert status() == binding.ATTN_OK
        model.same(cache)
        model.consistent()
        same_weights(weights, host)

    cut()
    one, T = i32([1, 1, 1]), [6, 1, 9]
    tq, tk, tv, tlse = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((3, Hq, D), (3, Hkv, D), (3, Hkv, D), (1,)))
    out, tlse = torch.empty_like(tq), torch.empty((Hq, 3), device="cuda")
    st, nbytes = binding.attn_fwd_tree_workspace(3, D)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    cu1 = offsets([1, 1, 1])

    def step():
        binding.kv_extend(cache, one, seqs=rows)
        binding.kv_append(cache, tk, tv, cu1, seqs=rows)
        binding.attention_tree(tq, cache, cu1, seqs=rows, out=out, lse_out=tlse, workspace=ws)
        binding.kv_weigh(cache, weights, tq, tlse, cu1, seqs=rows)
        binding.kv_evict(cache, rows, weights, **keeps)

    graph = None
    for turn in range(5):
        y = queries(3, Hq + 2 * Hkv, D, dtype, 100 + turn)
        tq.copy_(y[:, :Hq]), tk.copy_(y[:, Hq:Hq + Hkv]), tv.copy_(y[:, Hq + Hkv:])
        before = binding.KVPages(cache.k.clone(), cache.v.clone(), cache.table.clone(), cache.lens.clone(), cache.refs.clone())
        old = weights.clone()
        if turn < 2:
            step()
        else:
            if graph is None:
                s = torch.cuda.Stream()
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=s):
                        step()
                torch.cuda.current_stream().wait_stream(s)
            graph.replay()
        assert status() == binding.ATTN_OK
        # the same step on the copy, call by call, each held against its definition
        binding.kv_extend(before, one, seqs=rows)
        binding.kv_append(before, tk, tv, cu1, seqs=rows)
        check(tq, before, out, tlse, range(3), [[-1]] * 3, dtype, scale)
        grown = before.lens.tolist()[:3]
        for s in range(3):
            n = grown[s]
            want, tol = weigh_plain(tq[s:s + 1], tlse[:, s:s + 1], gather(before, s)[0], 1, scale)
            want[:, :n - 1] += old[0, s, :, :n - 1].double().cpu()
            tol += F * want
            old[0, s, :, :n] = want.float().cuda()
            bound = tol
            if n <= 80:  # not cut
                close(weights[0, s, :, :n], want, bound, f"turn {turn}, sequence {s}")
            else:
                assert int(cache.lens[s]) == 80
                # what is kept is a part of what was, in order
                for h in range(Hkv):
                    got = weights[0, s, h, :80].double().cpu()
                    near = (got[:, None] - want[h][None]).abs() <= bound[h][None]
                    assert bool(near.any(1).all())
                assert bool((weights[0, s, :, 80:] == 0).all())
    # drafted trees over the cut cache, and with a window over it
    par = trees(T, 31)
    binding.kv_extend(cache, i32(T), seqs=rows)
    z = queries(sum(T), Hq + 2 * Hkv, D, dtype, 33)
    binding.kv_append(cache, z[:, Hq:Hq + Hkv], z[:, Hq + Hkv:], offsets(T), seqs=rows)
    flat = i32([t for p in par for t in p])
    o, lse = binding.attention_tree(z[:, :Hq], cache, offsets(T), seqs=rows, parents=flat)
    assert status() == binding.ATTN_OK
    check(z[:, :Hq], cache, o, lse, range(3), par, dtype, scale)
    path = torch.full((3, 2), -1, dtype=torch.int32)
    path[:, 0] = 0
    binding.kv_accept(cache, offsets(T), path.cuda(), i32([1, 1, 1]), seqs=rows)
    assert cache.lens.tolist()[:3] == [81, 81, 81] and status() == binding.ATTN_OK
    cut()
    binding.kv_free(cache, rows)
    assert status() == binding.ATTN_OK and bool((cache.refs == 0).all())


@pytest.mark.parametrize("T", [32, 20])
def test_units_of_one_row_tile_hand_their_sums_over_in_turn(T):
    """Thousands of units with one row tile each, in which both warpgroups of a key tile have columns:
    every call ends, and gives what the first gave."""
    lens = [2000 + 37 * i for i in range(16)]
    cache = build(lens, 64, 8, 128, "bf16", seed=31)
    q = queries(16 * T, 32, 128, "bf16", 32)
    lse = torch.full((32, 16 * T), 9.0, device="cuda")
    weights, first = cache.weights(), None
    for _ in range(40):
        binding.kv_weigh(cache, weights, q, lse, offsets([T] * 16), accumulate=False)
        first = weights.clone() if first is None else first
        assert torch.equal(weights, first)
    assert status() == binding.ATTN_OK
    for s in (0, 15):
        want, tol = weigh_plain(q[s * T:s * T + T], lse[:, s * T:s * T + T], gather(cache, s)[0], T, 1 / math.sqrt(128))
        close(weights[0, s, :, :lens[s]], want, tol, f"sequence {s}")


def test_whole_prompts_of_many_units():
    """More units than CTAs, dealt by the work that they have."""
    lens = [1500, 33, 900, 1, 1200, 700, 128, 1024, 513, 256, 90, 400]
    Hq, Hkv, D = 16, 8, 64
    cache = build(lens, 32, Hkv, D, "f16", seed=51)
    q, scale, a = queries(sum(lens), Hq, D, "f16", 52), 0.125, 0
    lse = torch.empty((Hq, sum(lens)), device="cuda")
    for s, n in enumerate(lens):
        lse[:, a:a + n] = logsumexps(q[a:a + n], gather(cache, s)[0], n, scale)
        a += n
    weights = cache.weights() + 5
    binding.kv_weigh(cache, weights, q, lse, offsets(lens))
    assert status() == binding.ATTN_OK
    a = 0
    for s, n in enumerate(lens):
        want, tol = weigh_plain(q[a:a + n], lse[:, a:a + n], gather(cache, s)[0], n, scale)
        close(weights[0, s, :, :n], want, tol, f"prompt {s}")
        assert bool((weights[0, s, :, n:] == 5).all())
        a += n


@pytest.mark.parametrize("long,short,n_short,Hkv", [(1300, 200, 31, 12), (700, 100, 31, 16), (3000, 130, 20, 16)])
def test_large_and_small_units_share_the_first_round(long, short, n_short, Hkv):
    """Units of many row tiles beside so many of few that the CTAs' first ones are of both kinds, and several rounds follow."""
    lens, D = [long] + [short + i for i in range(n_short)], 64
    cache = build(lens, 64, Hkv, D, "bf16", seed=55)
    q, scale, a = queries(sum(lens), Hkv, D, "bf16", 56), 0.125, 0
    lse = torch.empty((Hkv, sum(lens)), device="cuda")
    for s, n in enumerate(lens):
        lse[:, a:a + n] = logsumexps(q[a:a + n], gather(cache, s)[0], n, scale)
        a += n
    weights = torch.full_like(cache.weights(), -3.0)
    binding.kv_weigh(cache, weights, q, lse, offsets(lens))
    assert status() == binding.ATTN_OK
    a = 0
    for s, n in enumerate(lens):
        want, tol = weigh_plain(q[a:a + n], lse[:, a:a + n], gather(cache, s)[0], n, scale)
        close(weights[0, s, :, :n], want, tol, f"prompt {s}")
        a += n


@pytest.mark.parametrize("layers,Hkv,n,page", [(1, 1, 300000, 1024), (20, 8, 40000, 256), (1, 2, 70000, 16)])
def test_eviction_from_very_long_sequences(layers, Hkv, n, page):
    """More positions than a cluster (of 8 blocks, of one) holds bits of at a time, with ties on the border."""
    sinks, heavy, recent, D = 5, 1234, 777, 64
    keep = sinks + heavy + recent
    cache = build([n], page, Hkv, D, "bf16", n_layers=layers, seed=61)
    weights = torch.floor(torch.rand(cache.weights().shape, device="cuda") ** 4 * 3000) / 3000
    k, v, w, table = cache.k.clone(), cache.v.clone(), weights[:, 0].clone(), cache.table.clone()
    binding.kv_evict(cache, i32([0]), weights, sinks=sinks, heavy=heavy, recent=recent)
    assert status() == binding.ATTN_OK and cache.lens.tolist() == [keep]
    best = torch.sort(w[:, :, sinks:n - recent], dim=-1, descending=True, stable=True).indices[:, :, :heavy] + sinks
    at = torch.arange(n, device="cuda").expand(layers, Hkv, n)
    src = torch.cat([at[:, :, :sinks], best.sort(-1).values, at[:, :, n - recent:]], -1)
    dst, row = at[:, :, :keep], table[0].long()
    L, H = torch.arange(layers, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[None, :, None]
    for old, new in ((k, cache.k), (v, cache.v)):
        old[L, row[dst // page], H, dst % page] = old[L, row[src // page], H, src % page]
        assert torch.equal(old.view(torch.int16), new.view(torch.int16))
    w2 = torch.zeros_like(w)
    w2[:, :, :keep] = torch.gather(w, 2, src)
    assert torch.equal(weights[:, 0, :, :n], w2[:, :, :n])
    used = -(-keep // page)
    assert torch.equal(cache.table[0, :used], table[0, :used]) and bool((cache.table[0, used:] == -1).all())
    assert int(cache.refs.sum()) == used


def test_a_wait_that_runs_out_ends_the_call_and_the_next_one_is_right():
    cache = build([900, 300], 64, 2, 128, "bf16", seed=71)
    T = [40, 3]
    q, lse = queries(43, 8, 128, "bf16", 72), torch.full((8, 43), 6.0, device="cuda")
    good, weights, lib = cache.weights(), cache.weights(), binding.load()
    binding.kv_weigh(cache, good, q, lse, offsets(T))
    o, _ = binding.attention_tree(q, cache, offsets(T), window=200, sinks=4)
    x = queries(300, 8, 128, "bf16", 73)
    p, _ = binding.attention_varlen(x, x[:, :2], x[:, 2:4], offsets([300]), window=40, sinks=4)
    assert status() == binding.ATTN_OK
    for call in (lambda: binding.kv_weigh(cache, weights, q, lse, offsets(T)),
                 lambda: binding.attention_tree(q, cache, offsets(T), window=200, sinks=4),
                 lambda: binding.attention_varlen(x, x[:, :2], x[:, 2:4], offsets([300]), window=40, sinks=4)):
        try:
            lib.attn_test_set_wait_timeout_ns(20_000_000)
            lib.attn_test_inject_stall(1)
            call()
        finally:
            lib.attn_test_inject_stall(0)
            lib.attn_test_set_wait_timeout_ns(0)
        assert status() == binding.ATTN_ERR_TIMEOUT
        call()
        assert status() == binding.ATTN_OK
    weights.zero_()
    binding.kv_weigh(cache, weights, q, lse, offsets(T))
    assert torch.equal(weights, good)
    assert torch.equal(o, binding.attention_tree(q, cache, offsets(T), window=200, sinks=4)[0])
    assert torch.equal(p, binding.attention_varlen(x, x[:, :2], x[:, 2:4], offsets([300]), window=40, sinks=4)[0])


def test_calls_on_two_streams_and_in_two_graphs():
    """Two caches at once, each on its own stream, and a graph of each replayed at once."""
    sides = []
    for seed in (81, 82):
        cache = build([700 + seed, 300, 500], 32, 2, 64, "f16", seed=seed, n_layers=2)
        q, lse = queries(30, 4, 64, "f16", seed), torch.full((4, 30), 5.5, device="cuda")
        weights, cu = cache.weights(), offsets([10, 10, 10])
        state = [x.clone() for x in (cache.k, cache.v, cache.table, cache.lens, cache.refs)]
        s = torch.cuda.Stream()

        def step(cache=cache, q=q, lse=lse, weights=weights, cu=cu, state=state):
            for x, y in zip((cache.k, cache.v, cache.table, cache.lens, cache.refs), state):
                x.copy_(y)
            for layer in (0, 1):
                binding.kv_weigh(cache, weights, q, lse, cu, layer=layer, accumulate=False)
            binding.kv_evict(cache, None, weights, sinks=3, heavy=100, recent=60)

        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in (cache.k, cache.v, cache.table, cache.lens, cache.refs, weights)]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
        sides.append((cache, weights, want, step, s, graph))
    torch.cuda.synchronize()
    for _ in range(10):
        for cache, weights, want, step, s, graph in sides:
            with torch.cuda.stream(s):
                step()
                graph.replay()
    torch.cuda.synchronize()
    assert status() == binding.ATTN_OK
    for cache, weights, want, step, s, graph in sides:
        for x, y in zip((cache.k, cache.v, cache.table, cache.lens, cache.refs, weights), want):
            assert torch.equal(x, y)
        assert cache.lens.tolist() == [163, 163, 163]
